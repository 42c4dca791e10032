"""The serving operators together with the compressed projections: the example's prompt and
verify steps against its plain computation."""

import pytest

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("requests,seed", [(6, 0), (1, 3), (17, 5)])
def test_verify_step_example(requests, seed):
    from examples import verify_step
    assert verify_step.main(requests, seed) < 2e-2


@pytest.mark.parametrize("path", ["first", "last"])
def test_verify_steps_return_their_pages(path):
    """Trees of 17 to 40 nodes, of which one or a few are kept, over more steps than the pool
    has pages for if each kept those of its dropped nodes: no page is lost or held twice."""
    import numpy as np
    import torch
    from examples import verify_step as e
    rng = np.random.default_rng(1)
    requests, steps = 5, 60
    s = e.Server(requests)
    dev = lambda a: torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")
    for _ in range(steps):
        nodes = rng.integers(17, 41, requests)
        cu = np.concatenate([[0], np.cumsum(nodes)])
        parents = np.concatenate([[-1] + [int(rng.integers(max(-1, i - 9), i)) for i in range(1, n)] for n in nodes])
        x = torch.zeros((int(cu[-1]), e.HIDDEN), dtype=torch.bfloat16, device="cuda")
        _, p = s.step(x, dev(nodes), parents=dev(parents))
        assert int(p.counts[2]) == 0
        lens = np.ones(requests, int) if path == "first" else np.minimum(nodes, 3)
        rows = [cu[r] + j for r in range(requests) for j in range(lens[r])]
        s.keep(p, torch.tensor(rows, device="cuda"), dev(lens))
        held, free = s.table[s.table >= 0].tolist(), s.free[int(s.head):].tolist()
        assert sorted(held + free) == list(range(e.BLOCKS))
    # at least one page a request and step would have been lost
    assert requests * steps > e.BLOCKS - len(held)
