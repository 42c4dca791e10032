"""The serving operators together with the compressed projections: the example's prompt and
verify steps against its plain computation."""

import pytest

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("requests,seed", [(6, 0), (1, 3), (17, 5)])
def test_verify_step_example(requests, seed):
    from examples import verify_step
    assert verify_step.main(requests, seed) < 2e-2
