"""Pins of the oracle of rotation, verification and page moves: closed forms, hand-worked cases,
and controls that a wrong definition would fail."""

import numpy as np

from oracle import serving


def test_rotation_is_a_turn():
    rng = np.random.default_rng(0)
    x = rng.normal(size=(3, 2, 8))
    freqs = np.array([1.0, 0.1, 0.01, 0.001])
    for inter in (False, True):
        assert np.allclose(serving.rope(x, [0, 0, 0], freqs, interleaved=inter), x)
        y = serving.rope(x, [7, 70, 700], freqs, interleaved=inter)
        assert np.allclose(np.linalg.norm(y, axis=2), np.linalg.norm(x, axis=2))
        # turning by a and b is turning by a + b; products hang on the distance only
        assert np.allclose(serving.rope(y, [5, 5, 5], freqs, interleaved=inter),
                           serving.rope(x, [12, 75, 705], freqs, interleaved=inter))
        one = lambda p: serving.rope(x, [p] * 3, freqs, interleaved=inter)
        assert np.allclose((one(3)[0] * one(9)[1]).sum(1), (one(103)[0] * one(109)[1]).sum(1))
    # a quarter turn of one pair, the rest left as it is
    y = serving.rope(np.arange(6.0).reshape(1, 1, 6), [1], [np.pi / 2])
    assert np.allclose(y, [[[-1, 0, 2, 3, 4, 5]]])
    y = serving.rope(np.arange(6.0).reshape(1, 1, 6), [1], [0, np.pi], interleaved=True)
    assert np.allclose(y, [[[0, 1, -2, -3, 4, 5]]])


def test_norm_by_hand():
    y = serving.rope([[[3.0, 4.0, 0.0, 0.0]]], [0], [], weight=[1, 2, 3, 4], eps=0.0)
    assert np.allclose(y, [[[3 / 2.5, 8 / 2.5, 0, 0]]])


def test_verify_by_hand():
    logits = np.log(np.array([[0.5, 0.3, 0.2], [0.1, 0.6, 0.3], [0.25, 0.25, 0.5]]))
    # a chain: token 0 after row 0 (p = 0.5), token 1 after row 1 (p = 0.6)
    run = lambda u, s, **kw: serving.verify(logits, [9, 0, 1], np.array([0.0, u[0], u[1]]), s, **kw)
    assert run((0.49, 0.59), 0.3) == ([0, 1, 2], 1) and run((0.49, 0.59), 0.51) == ([0, 1, 2], 2)
    assert run((0.51, 0.0), 0.59) == ([0], 1) and run((0.51, 0.0), 0.61) == ([0], 2)
    assert run((0.49, 0.61), 0.24) == ([0, 1], 0) and run((0.49, 0.61), 0.26) == ([0, 1], 2)
    # two children of row 0: the second is looked at with what the first left, 0.3 of 0.5
    tree = lambda u, v, s: serving.verify(logits, [9, 0, 1], np.array([0.0, u, v]), s, parents=[-1, 0, 0])
    assert tree(0.6, 0.59, 0.0) == ([0, 2], 0) and tree(0.6, 0.61, 0.0) == ([0], 2)
    # with the draft's probabilities: accepted with p / q = 0.5 / 0.8; else from max(p - q, 0) = 0, 0.2, 0.1
    q = np.array([[0.8, 0.1, 0.1]] * 3, np.float32)
    assert run((0.62, 0.9), 0.0, probs=q)[0][:2] == [0, 1]
    assert run((0.63, 0.0), 0.66, probs=q) == ([0], 1) and run((0.63, 0.0), 0.67, probs=q) == ([0], 2)
    # the most likely tokens
    assert run((0.9, 0.9), 0.0, temperature=0.0) == ([0, 1, 2], 2)
    assert serving.verify(logits, [9, 1, 1], np.zeros(3), 0.0, temperature=-1.0) == ([0], 0)


def test_verify_keeps_the_targets_distribution():
    """By enumeration: over a fine grid of uniform numbers, what comes first is distributed as p."""
    p, q = np.array([0.5, 0.3, 0.2]), np.array([0.2, 0.2, 0.6], np.float32)
    grid = (np.arange(40) + 0.5) / 40
    for probs in (None, np.tile(q, (2, 1))):
        got = np.zeros(3)
        for x in range(3):
            weight = q[x] if probs is not None else 1 / 3  # any choice of a given draft will do
            for u in grid:
                for s in grid:
                    path, token = serving.verify(np.log(np.tile(p, (2, 1))), [0, x], [0, u], s, probs=probs)
                    got[x if len(path) > 1 else token] += weight / 1600
        assert np.allclose(got, p, atol=0.02), got


def test_verify_of_odd_rows():
    bad = np.array([[0.0, np.nan], [0.0, 0.0]])
    assert serving.verify(bad, [0, 0], [0, 0.0], 0.5) == ([0], -1)
    assert serving.verify(np.full((1, 2), -np.inf), [0], [0], 0.5) == ([0], -1)
    assert serving.verify(np.zeros((0, 2)), [], [], 0.5) == ([], -1)


def test_keep_by_hand():
    # pages of 8; 6 tokens cached, 5 new ones in pages 4 and 7; rows 0, 2, 3 stay: 9 tokens, two pages
    table = [[4, 7, -1]]
    slots = [4 * 8 + 6, 4 * 8 + 7, 7 * 8, 7 * 8 + 1, 7 * 8 + 2]
    moves, lens, free, t, counts = serving.page_keep([0, 2, 3, -1, -1], [3], [6], [0, 5], slots, [1, 4, 7, 2], 3, table,
                                                     8, 8)
    assert moves == [(56, 39), (57, 56)] and lens.tolist() == [9]
    assert t.tolist() == table and counts.tolist() == [3, 0]
    # only row 0 stays: page 7 goes back, in front of the head
    _, lens, free, t, counts = serving.page_keep(None, [1], [6], [0, 5], slots, [1, 4, 9, 2], 3, table, 8, 8)
    assert lens.tolist() == [7] and t.tolist() == [[4, -1, -1]] and counts.tolist() == [2, 1]
    assert free.tolist() == [1, 4, 7, 2]


def test_fork_and_free_by_hand():
    table = [[4, 7, -1], [-1, -1, -1], [-1, -1, -1]]
    copies, lens, t, shares, counts = serving.page_fork([0, 0], [1, 2], [11, 0, 0], [9, 4, 7, 2, 3], 3, table,
                                                        [0] * 10, 8, 10)
    assert copies == [(7, 2, 3), (7, 3, 3)] and lens.tolist() == [11] * 3 and counts.tolist() == [5, 0]
    assert t.tolist() == [[4, 7, -1], [4, 2, -1], [4, 3, -1]] and shares.tolist() == [0] * 4 + [2] + [0] * 5
    lens, free, t, shares, counts = serving.page_free([0, 2, 0], lens, [9, 4, 7, 2, 3], 5, t, shares, 8, 10)
    assert free.tolist() == [9, 4, 7, 3, 7] and counts.tolist() == [3, 2] and lens.tolist() == [0, 11, 0]
    assert shares.sum() == 0 and t.tolist() == [[-1] * 3, [4, 2, -1], [-1] * 3]
    _, free, t, _, counts = serving.page_free([1], lens, free, 3, t, shares, 8, 10)
    assert counts.tolist() == [1, 2] and free.tolist() == [9, 2, 4, 3, 7]


def _odd_trees():
    """Trees of the page plan whose nodes do not all get a slot: 100 nodes in one mask word, a bad link at a
    page's start and inside one, one whose nodes past the first all hang off a bad link; and a plain one."""
    chain = [-1] + list(range(99))
    bent = [-1] + list(range(39))
    bent[11], bent[27] = 11, -7  # node 11 lies first in a page of 16 behind 5 cached tokens
    cut = [-1, 1] + list(range(1, 29))
    new, ctx = [100, 40, 30, 20], [0, 5, 16, 9]
    return ctx, new, np.array(chain + bent + cut + [-1] + list(range(19)))


def odd_step(block=16, spare=3):
    """A step of such trees, planned by the oracle: what the plan left, and each request's tokens with a slot."""
    ctx, new, parents = _odd_trees()
    have = [-(-c // block) for c in ctx]
    pages = sum(-(-(c + n) // block) for c, n in zip(ctx, new))
    blocks = pages + spare
    ids = np.random.default_rng(3).permutation(blocks)
    table, at = np.full((4, 9), -1), 0
    for b, h in enumerate(have):
        table[b, :h] = ids[at:at + h]
        at += h
    table, cu, slots, _, _, counts = serving.page_plan(ctx, new, ids, at, table, block, blocks, sum(new), parents, 1)
    assert counts.tolist() == [sum(new), pages, 0]
    return dict(ctx=np.array(ctx), new=np.array(new), parents=parents, cu=cu, table=table, slots=slots, free=ids,
                first=at, head=int(counts[1]), blocks=blocks, block=block)


def held_or_free(d, table, lens, free, head):
    """Every page is in one request's columns up to its length, or in the list; no column past a length is set."""
    held = [int(p) for row, n in zip(table, lens) for p in row[:-(-int(n) // d["block"])]]
    past = [int(p) for row, n in zip(table, lens) for p in row[-(-int(n) // d["block"]):]]
    assert set(past) <= {-1}
    assert sorted(held + [int(p) for p in free[head:]]) == list(range(d["blocks"]))


def test_keep_returns_pages_of_tokens_without_a_slot():
    d = odd_step()
    assert (d["slots"][64:100] == -1).all() and d["slots"][111] == -1
    for kept in ([1, 1, 1, 1], [40, 11, 1, 20], [64, 1, 0, 0]):
        moves, lens, free, table, counts = serving.page_keep(
            None, kept, d["ctx"], d["cu"], d["slots"], d["free"], d["head"], d["table"], d["block"], d["blocks"])
        assert lens.tolist() == (d["ctx"] + kept).tolist() and moves == []
        held_or_free(d, table, lens, free, int(counts[0]))


def test_keep_ends_a_path_at_a_row_without_a_slot():
    """What was never stored is not counted: a node past the mask, one behind a bad link, a place on the path
    that has no slot."""
    d = odd_step()
    keep = lambda path, kept: serving.page_keep(path, kept, d["ctx"], d["cu"], d["slots"], d["free"], d["head"],
                                                d["table"], d["block"], d["blocks"])
    _, lens, free, table, counts = keep(None, [100, 40, 30, 20])
    assert lens.tolist() == [64, 5 + 11, 16 + 1, 9 + 20]
    held_or_free(d, table, lens, free, int(counts[0]))
    # request 0: rows 0, 60, 63, 64; request 1: rows 0, 5, 11 (no slot); request 3: rows 0, 3, 4
    path = np.full(190, -1)
    path[:4], path[100:104], path[140:142], path[170:173] = [0, 60, 63, 64], [0, 5, 11, 12], [0, 1], [0, 3, 4]
    moves, lens, free, table, counts = keep(path, [4, 4, 2, 3])
    s = d["slots"]
    assert lens.tolist() == [3, 5 + 2, 16 + 1, 9 + 3]
    assert moves == [(s[60], s[1]), (s[63], s[2]), (s[105], s[101]), (s[173], s[171]), (s[174], s[172])]
    held_or_free(d, table, lens, free, int(counts[0]))


def test_verify_at_an_infinite_temperature():
    """All tokens weigh the same but those of -inf."""
    row = np.array([[-np.inf, 3.0, -3.4e38, 7.0, -np.inf]])
    got = [serving.verify(row, [0], [0.0], s, temperature=np.inf) for s in (0.0, 0.33, 0.34, 0.66, 0.67)]
    assert got == [([0], 1), ([0], 1), ([0], 2), ([0], 2), ([0], 3)]
