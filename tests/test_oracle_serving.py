"""Pins of the serving oracle: hand-worked plans, closed forms of attention and
adapters, and controls that a wrong mask or a lost page would fail."""

import numpy as np
import pytest

from oracle import serving


def test_plan_by_hand():
    # pages of 8: request 0 holds 7 (1 page) and brings 2 (crosses into a fresh page),
    # request 1 holds 8 exactly and brings 1, request 2 brings nothing
    table = [[5, -1, -1], [2, -1, -1], [9, 4, -1]]
    table, cu, slots, pos, mask, counts = serving.page_plan(
        [7, 8, 16], [2, 1, 0], [30, 31, 32, 33], 1, table, 8, 40, 4)
    assert table.tolist() == [[5, 31, -1], [2, 32, -1], [9, 4, -1]]
    assert cu.tolist() == [0, 2, 3, 3]
    assert slots.tolist() == [5 * 8 + 7, 31 * 8, 32 * 8, -1]
    assert pos.tolist() == [7, 8, 8, -1]
    assert mask is None and counts.tolist() == [3, 3, 0]


def test_plan_refusals_by_hand():
    # two pages left: request 0 takes both, 1 needs one and is refused, 2 needs none
    table, cu, slots, pos, _, counts = serving.page_plan(
        [0, 8, 3], [16, 1, 1], [1, 2], 0, [[-1, -1], [3, -1], [4, -1]], 8, 10, 18)
    assert counts.tolist() == [18, 2, 1]
    assert slots[16] == -1 and pos[16] == 8 and slots[17] == 4 * 8 + 3
    # a table too narrow, and rows that do not fit
    _, _, slots, _, _, counts = serving.page_plan([15], [2], [1, 2], 0, [[3, 4]], 8, 10, 2)
    assert counts.tolist() == [2, 0, 1] and slots.tolist() == [-1, -1]
    _, cu, slots, _, _, counts = serving.page_plan([0, 0], [2, 2], [1, 2], 0, [[-1], [-1]], 8, 10, 3)
    assert cu.tolist() == [0, 2, 3] and counts.tolist() == [4, 1, 1]
    assert slots.tolist() == [8, 9, -1]


def test_plan_tree_by_hand():
    #      0        3
    #     / \
    #    1   2 -> 4
    parents = [-1, 0, 0, -1, 2]
    _, _, slots, pos, mask, _ = serving.page_plan([10], [5], [7], 0, [[1, 2]], 8, 10, 5, parents, 1)
    assert mask[:, 0].tolist() == [0b1, 0b11, 0b101, 0b1000, 0b10101]
    assert pos.tolist() == [10, 11, 11, 10, 12]
    assert slots.tolist() == [18, 19, 20, 21, 22]
    # a parent that is not below its child spoils the child and its descendants
    _, _, slots, pos, mask, _ = serving.page_plan([10], [5], [7], 0, [[1, 2]], 8, 10, 5, [-1, 0, 2, -1, 2], 1)
    assert mask[:, 0].tolist() == [1, 3, 0, 8, 0] and pos.tolist() == [10, 11, -1, 10, -1]
    assert slots.tolist() == [18, 19, -1, 21, -1]
    assert (serving.pack_mask(serving.ancestors(parents), 1)[:, 0] == [1, 3, 5, 8, 21]).all()


def test_attention_of_equal_scores_is_a_mean():
    rng = np.random.default_rng(0)
    keys, values = rng.normal(size=(9, 2, 4)), rng.normal(size=(9, 2, 4))
    seen = np.array([[1, 0, 0], [1, 1, 0], [0, 0, 0]], bool)
    out, size = serving.tree_attention(np.zeros((3, 4, 4)), keys, values, 6, seen, 0.5)
    for h in range(4):
        assert np.allclose(out[0, h], values[:7, h // 2].mean(0))
        assert np.allclose(out[1, h], values[:8, h // 2].mean(0))
        assert np.allclose(out[2, h], values[:6, h // 2].mean(0))
    assert (size >= np.abs(out) - 1e-12).all()
    # nothing seen: zero
    out, _ = serving.tree_attention(np.ones((3, 4, 4)), keys[6:], values[6:], 0, seen, 0.5)
    assert (out[2] == 0).all() and np.allclose(out[0, 1], values[6, 0])


def test_attention_of_two_keys_is_a_logistic():
    q = np.array([[[2.0, 0.0]]])
    keys = np.array([[[1.5, 3.0]], [[0.5, -1.0]]])
    values = np.array([[[1.0, 0.0]], [[0.0, 1.0]]])
    out, _ = serving.tree_attention(q, keys, values, 1, np.ones((1, 1), bool), 0.25)
    p = 1 / (1 + np.exp(-0.25 * 2.0 * (1.5 - 0.5)))
    assert np.allclose(out[0, 0], [p, 1 - p], rtol=1e-14)


def test_lora_by_hand():
    x = np.array([[1.0, 2.0], [3.0, -1.0], [1.0, 1.0]])
    a = np.array([[[1.0, 1.0]], [[2.0, 0.0]]])          # rank 1
    b = np.array([[[1.0], [0.0]], [[1.0], [-1.0]]])
    out, size = serving.lora_add(np.ones((3, 2)), x, a, b, [2.0, 0.5], [1, -1, 0], [0, 1, 2, 3])
    assert out.tolist() == [[2.0, 0.0], [1.0, 1.0], [5.0, 1.0]]
    assert size.tolist() == [[1.0, 1.0], [0.0, 0.0], [4.0, 0.0]]


@pytest.mark.parametrize("n", [1, 7, 70])
def test_ancestors_are_a_partial_order(n):
    rng = np.random.default_rng(n)
    parents = [-1] + [int(rng.integers(-1, i)) for i in range(1, n)]
    seen = serving.ancestors(parents)
    assert seen.diagonal().all() and not np.triu(seen, 1).any()
    for i in range(n):
        for j in np.nonzero(seen[i])[0]:
            assert (seen[i] >= seen[j]).all()   # transitive
    words = (n + 63) // 64
    packed = serving.pack_mask(seen, words)
    back = np.unpackbits(packed.view(np.uint8), axis=1, bitorder="little")[:, :n].astype(bool)
    assert (back == seen).all()
