"""Keeping, forking and freeing pages against the oracle: everything is copied or counted, so everything
is equal, and every cell that is not named stays as it was."""

import numpy as np
import pytest

import decode_gemm_tile_amd as dgt
from oracle import serving

pytestmark = pytest.mark.gpu


def _i32(a):
    import torch
    return torch.from_numpy(np.ascontiguousarray(np.asarray(a, np.int32))).to("cuda")


def _caches(seed, layers, blocks, heads, block, dim, dtype="bfloat16"):
    """Every bit pattern, NaNs too: copies are bit for bit."""
    import torch
    g = torch.Generator().manual_seed(seed)
    front = () if layers is None else (layers,)
    made = lambda *s: torch.randint(-2 ** 15, 2 ** 15, front + s, generator=g, dtype=torch.int16).view(getattr(torch, dtype))
    return made(blocks, heads, block, dim), made(blocks, heads, dim, block)


def _bits(t):
    import torch
    return t.cpu().view(torch.int16)


def _step(seed, ctx, new, block, extra=6, refuse=()):
    """Tables with the step's pages in them, slots as the plan leaves them, and a free list."""
    rng = np.random.default_rng(seed)
    ctx, new = np.asarray(ctx), np.asarray(new)
    pages = -(-(ctx + new) // block)
    blocks = int(pages.sum()) + extra
    ids, at = rng.permutation(blocks), 0
    table = np.full((len(ctx), int(pages.max(initial=0)) + 2), -1)
    for b, p in enumerate(pages):
        table[b, :p] = ids[at:at + p]
        at += p
    slots = [table[b, (c + i) // block] * block + (c + i) % block if b not in refuse else -1
             for b, (c, n) in enumerate(zip(ctx, new)) for i in range(n)]
    free = np.concatenate([ids[:at], ids[at:]])  # those taken lie in front of the head
    return dict(ctx=ctx, new=new, cu=np.concatenate([[0], np.cumsum(new)]), table=table,
                slots=np.array(slots, int), free=free, head=at, blocks=blocks, block=block)


def _paths(seed, new, kept):
    rng = np.random.default_rng(seed)
    path = np.full(int(sum(new)), -1)
    at = 0
    for n, k in zip(new, kept):
        k = min(max(k, 0), n)
        if k:
            path[at:at + k] = np.concatenate([[0], 1 + np.sort(rng.choice(n - 1, k - 1, replace=False))]) if k > 1 else [0]
        at += n
    return path


def _keep(d, path, kept, layers, heads, dim, dtype="bfloat16", in_place=True):
    import torch
    k, v = _caches(3, layers, d["blocks"], heads, d["block"], dim, dtype)
    kd, vd, table, free, ctx = k.cuda(), v.cuda(), _i32(d["table"]), _i32(d["free"]), _i32(d["ctx"])
    counts = torch.tensor([99, d["head"], 0], dtype=torch.int32, device="cuda")
    lens = None if in_place else torch.zeros_like(ctx)
    got = dgt.dgt_page_keep(_i32(kept), ctx, _i32(d["cu"]), _i32(d["slots"]), free, counts[1:2], table, kd, vd,
                            path=None if path is None else _i32(path), lens=lens,
                            counts=counts[1:] if in_place else None)
    moves, ref_lens, ref_free, ref_table, ref_counts = serving.page_keep(
        path, kept, d["ctx"], d["cu"], d["slots"], d["free"], d["head"], d["table"], d["block"], d["blocks"])
    assert got.tolist() == ref_counts.tolist()
    assert (ctx if in_place else lens).tolist() == ref_lens.tolist()
    assert in_place or ctx.tolist() == list(d["ctx"])
    assert np.array_equal(table.cpu().numpy(), ref_table) and np.array_equal(free.cpu().numpy(), ref_free)
    k0, v0 = (_bits(k).clone(), _bits(v).clone())
    k0, v0 = (x if layers is not None else x[None] for x in (k0, v0))
    ks, vs = k0.clone(), v0.clone()
    b = d["block"]
    for src, dst in moves:
        k0[:, dst // b, :, dst % b] = ks[:, src // b, :, src % b]
        v0[:, dst // b, :, :, dst % b] = vs[:, src // b, :, :, src % b]
    assert torch.equal(_bits(kd).view(k0.shape), k0) and torch.equal(_bits(vd).view(v0.shape), v0)


KEEPS = [  # ctx, new, kept, layers, heads, dim, block
    ([0], [1], [1], None, 1, 8, 8),
    ([15], [5], [2], None, 2, 64, 16),
    ([3, 40, 0], [9, 30, 17], [3, 8, 17], 2, 2, 80, 16),
    ([100, 0, 31, 7], [61, 0, 2, 33], [5, 0, 0, 20], 3, 1, 128, 32),
    ([5] * 300, [4] * 300, [i % 5 for i in range(300)], None, 1, 64, 8),
    ([1000], [300], [40], 1, 2, 256, 64),
    ([12, 9], [90, 50], [90, 49], 2, 3, 40, 8),
    ([7], [20], [6], 1, 1, 1024, 1024),
    ([2], [40], [1000], 1, 1, 24, 16),
]


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("i", range(len(KEEPS)))
def test_keep_against_oracle(i, in_place):
    ctx, new, kept, layers, heads, dim, block = KEEPS[i]
    d = _step(i, ctx, new, block)
    _keep(d, _paths(i, new, kept), kept, layers, heads, dim, in_place=in_place)
    _keep(d, None, kept, layers, heads, dim, "float16", in_place=in_place)


def test_keep_of_refused_requests():
    """A request that the plan refused has no slots: it keeps nothing and returns nothing."""
    d = _step(20, [10, 20, 30], [9, 9, 9], 8, refuse=(1,))
    _keep(d, _paths(20, d["new"], [4, 4, 4]), [4, 4, 4], 2, 2, 64)


def test_keep_of_paths_that_are_none():
    """Indexes out of range, or behind their own place, leave the place; counts are cut; slots outside the
    pool are passed over."""
    d = _step(21, [10, 20, 3], [20, 40, 8], 8)
    path = _paths(21, d["new"], [5, 12, 4])
    path[2], path[23], path[61] = 2 ** 31 - 1, -5, 0
    d["slots"][path[3]] = 2 ** 30
    _keep(d, path, [5, 12, -4], 1, 2, 64)


def test_keep_with_a_list_that_is_too_short_in_front():
    """More pages than the list has given out: the first of them are not returned."""
    import torch
    d = _step(22, [0, 0], [64, 64], 8)
    free = _i32(d["free"])
    table = _i32(d["table"])
    k, v = (x.cuda() for x in _caches(1, None, d["blocks"], 1, 8, 8))
    whole = torch.full((len(d["free"]) + 2,), 77, dtype=torch.int32, device="cuda")
    whole[1:-1] = free
    counts = dgt.dgt_page_keep(_i32([1, 1]), _i32(d["ctx"]), _i32(d["cu"]), _i32(d["slots"]), whole[1:-1], _i32([5]),
                               table, k, v)
    assert counts.tolist() == [0, 14] and whole[0] == 77 and whole[-1] == 77
    assert whole[1:6].tolist() == d["table"][1, 3:8].tolist() and whole[6:-1].tolist() == d["free"][5:].tolist()


def _fork(d, src, dst, lens, layers, heads, dim, shares=None, dtype="bfloat16"):
    import torch
    k, v = _caches(4, layers, d["blocks"], heads, d["block"], dim, dtype)
    shares = np.zeros(d["blocks"], int) if shares is None else shares
    kd, vd, table, free = k.cuda(), v.cuda(), _i32(d["table"]), _i32(d["free"])
    ls, sh = _i32(lens), _i32(shares)
    counts = torch.tensor([99, d["head"], 7], dtype=torch.int32, device="cuda")
    got = dgt.dgt_page_fork(_i32(src), _i32(dst), ls, free, counts[1:2], table, sh, kd, vd, counts=counts[1:])
    copies, ref_lens, ref_table, ref_shares, ref_counts = serving.page_fork(
        src, dst, lens, d["free"], d["head"], d["table"], shares, d["block"], d["blocks"])
    assert got.tolist() == ref_counts.tolist() and ls.tolist() == ref_lens.tolist()
    assert np.array_equal(table.cpu().numpy(), ref_table) and sh.tolist() == ref_shares.tolist()
    assert free.tolist() == list(d["free"])
    k0, v0 = _bits(k).clone(), _bits(v).clone()
    k0, v0 = (x if layers is not None else x[None] for x in (k0, v0))
    for a, b, n in copies:
        k0[:, b, :, :n], v0[:, b, :, :, :n] = k0[:, a, :, :n].clone(), v0[:, a, :, :, :n].clone()
    assert torch.equal(_bits(kd).view(k0.shape), k0) and torch.equal(_bits(vd).view(v0.shape), v0)
    return ref_table, ref_lens, ref_shares, int(ref_counts[0])


def _requests(seed, lens, empty, block, extra=20):
    d = _step(seed, lens, [0] * len(lens), block, extra=extra)
    d["table"] = np.concatenate([d["table"], np.full((empty, d["table"].shape[1]), -1)])
    return d, list(lens) + [0] * empty


FORKS = [  # lens, src, dst, layers, heads, dim, block
    ([1], [0], [1], None, 1, 8, 8),
    ([16], [0, 0], [2, 1], None, 2, 64, 16),
    ([17, 5, 32], [0, 1, 2, 0, 1], [3, 4, 5, 6, 7], 2, 2, 80, 16),
    ([1000, 3], [0] * 6 + [1] * 2, [2, 3, 4, 5, 6, 7, 8, 9], 3, 1, 128, 64),
    ([700], [0], [1], 1, 2, 256, 1024),
    ([9] * 100, list(range(100)), list(range(100, 200)), None, 1, 64, 8),
]


@pytest.mark.parametrize("i", range(len(FORKS)))
def test_fork_against_oracle(i):
    lens, src, dst, layers, heads, dim, block = FORKS[i]
    d, lens = _requests(i, lens, max(dst) + 1 - len(lens), block, extra=len(src) + 3)
    _fork(d, src, dst, lens, layers, heads, dim, dtype=["bfloat16", "float16"][i % 2])


def test_forks_that_are_refused():
    """Rows out of range, sources that are empty, destinations that are not or are named twice, a source whose
    pages the table does not hold, a list that runs out."""
    d, lens = _requests(30, [20, 33, 8, 7], 9, 8, extra=3)
    src = [0, -1, 0, 99, 5, 1, 1, 0, 2, 0, 3, 1]
    dst = [4, 5, 99, 6, 7, 2, 4, 5, 6, -1, 8, 9]
    _fork(d, src, dst, lens, 2, 1, 64)
    lens[3] = 2 ** 31 - 1
    _fork(d, src, dst, lens, None, 1, 64)
    d["head"] = len(d["free"])  # nothing left: only whole pages can be forked
    _fork(d, src, dst, lens, None, 1, 64)
    d["table"][0, 1] = -1       # a page that is missing
    d["head"] = len(d["free"]) - 3
    _fork(d, src, dst, lens, None, 1, 64)


def _free(rows, lens, d, shares, ws=None):
    import torch
    table, free, ls, sh = _i32(d["table"]), _i32(d["free"]), _i32(lens), _i32(shares)
    head = torch.tensor([d["head"], 0], dtype=torch.int32, device="cuda")
    got = dgt.dgt_page_free(_i32(rows), ls, free, head[:1], table, sh, d["block"], counts=head, ws=ws)
    ref_lens, ref_free, ref_table, ref_shares, ref_counts = serving.page_free(
        rows, lens, d["free"], d["head"], d["table"], shares, d["block"], d["blocks"])
    assert got.tolist() == ref_counts.tolist() and ls.tolist() == ref_lens.tolist()
    assert free.tolist() == ref_free.tolist() and sh.tolist() == ref_shares.tolist()
    assert np.array_equal(table.cpu().numpy(), ref_table)
    return ref_table, ref_lens, ref_shares, ref_free, int(ref_counts[0])


def test_free_against_oracle():
    import torch
    d, lens = _requests(40, [100, 1, 0, 640, 33], 3, 16)
    ws = dgt.alloc_workspace(dgt.dgt_page_free_workspace(d["blocks"]))
    _free([3, 0, 3, -1, 8, 2, 0, 2 ** 31 - 1], lens, d, np.zeros(d["blocks"], int), ws)
    assert not bool(ws.any())
    _free([], lens, d, np.zeros(d["blocks"], int), ws)
    _free(list(range(8)), lens, d, np.zeros(d["blocks"], int))


def test_fork_and_free_in_turn():
    """Forks of forks, freed in different orders: a page goes back with its last holder, once."""
    import torch
    rng = np.random.default_rng(5)
    for order in range(4):
        d, lens = _requests(50 + order, [45, 16, 130], 6, 16)
        start = set(d["free"][d["head"]:].tolist())
        table, lens, shares, head = _fork(d, [0, 2, 1], [3, 4, 5], lens, 1, 1, 64)
        d = dict(d, table=table, head=head)
        table, lens, shares, head = _fork(d, [3, 3, 2], [6, 7, 8], lens, 1, 1, 64, shares)
        d = dict(d, table=table, head=head)
        rows = rng.permutation(9)
        for part in (rows[:4], rows[4:5], rows[5:]):
            table, lens, shares, free, head = _free(part.tolist(), lens, d, shares)
            d = dict(d, table=table, free=free, head=head)
        assert head == 0 and sorted(free.tolist()) == list(range(d["blocks"])) and not shares.any()
        assert start <= set(free.tolist())


def test_many_requests_and_pages():
    """8192 rows; more pages than one round of the collecting workgroup looks at."""
    d, lens = _requests(60, [9] * 4000, 4192, 8, extra=4100)
    table, lens, shares, head = _fork(d, list(range(4000)), list(range(4000, 8000)), lens, None, 1, 8)
    d = dict(d, table=table, head=head)
    _free(list(range(0, 8192, 3)), lens, d, shares)
    d, lens = _requests(61, [70000 * 8], 0, 8, extra=1)
    _free([0], lens, d, np.zeros(d["blocks"], int))


def test_captured_steps_in_fixed_buffers():
    """Plan, keep, fork and free recorded once and replayed: the list's head goes from one to the next within
    one array, and no page is lost or held twice."""
    import torch
    requests, block, blocks, width = 4, 8, 200, 20
    table = torch.full((6, width), -1, dtype=torch.int32, device="cuda")
    lens = torch.zeros(6, dtype=torch.int32, device="cuda")
    new, kept = _i32([5, 9, 1, 12, 0, 0]), _i32([2, 9, 1, 3, 0, 0])
    free = torch.randperm(blocks, dtype=torch.int32).cuda()
    shares = torch.zeros(blocks, dtype=torch.int32, device="cuda")
    plan = dgt.PagePlan.empty(6, 27)
    plan.counts.zero_()
    head = plan.counts[1:2]
    k, v = (x.cuda() for x in _caches(1, 2, blocks, 1, block, 16))
    path = _i32(_paths(3, [5, 9, 1, 12], [2, 9, 1, 3]))
    src, dst, ws = _i32([0, 3]), _i32([4, 5]), dgt.alloc_workspace(dgt.dgt_page_free_workspace(blocks))
    counts = torch.zeros(2, dtype=torch.int32, device="cuda")

    def step():
        dgt.dgt_page_plan(lens, new, free, head, table, block, blocks, 27, out=plan)
        dgt.dgt_page_keep(kept, lens, plan.cu, plan.slots, free, head, table, k, v, path=path, counts=counts)
        dgt.dgt_page_fork(src, dst, lens, free, counts[:1], table, shares, k, v, counts=counts)
        dgt.dgt_page_free(dst, lens, free, counts[:1], table, shares, block, counts=counts, ws=ws)
        torch.add(counts[:1], 0, out=head)

    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(8):
        graph.replay()
        torch.cuda.synchronize()
        assert lens.tolist() == [2 * (i + 2), 9 * (i + 2), i + 2, 3 * (i + 2), 0, 0]
        held = table[table >= 0].tolist()
        assert sorted(held + free[int(head):].tolist()) == list(range(blocks)) and not bool(shares.any())


def test_empty_calls():
    import torch
    k, v = (x.cuda() for x in _caches(1, None, 3, 1, 8, 8))
    none, head = torch.zeros(0, dtype=torch.int32, device="cuda"), _i32([1])
    table, free, shares = torch.zeros((0, 4), dtype=torch.int32, device="cuda"), _i32([0, 1, 2]), _i32([0, 0, 0])
    assert dgt.dgt_page_keep(none, none, _i32([0]), none, free, head, table, k, v).tolist() == [1, 0]
    assert dgt.dgt_page_fork(none, none, none, free, head, table, shares, k, v).tolist() == [1, 0]
    assert dgt.dgt_page_free(none, none, free, head, table, shares, 8).tolist() == [1, 0]


@pytest.mark.parametrize("many", [1, 70])
@pytest.mark.parametrize("kept", [[1, 1, 1, 1], [40, 11, 1, 20], [64, 1, 0, 0]])
def test_keep_returns_pages_of_tokens_without_a_slot(kept, many):
    """The plan takes pages for every node, also for one past the mask or behind a bad link, which gets no
    slot: after the keep each page is held or free.  (70 steps' requests in one: more than one round.)"""
    import torch
    from tests.test_oracle_step import held_or_free, odd_step
    d = odd_step()
    shift = lambda x: np.concatenate([np.where(np.asarray(x) >= 0, np.asarray(x) + i * d["blocks"], -1)
                                      for i in range(many)])
    ctx, new, parents = np.tile(d["ctx"], many), np.tile(d["new"], many), np.tile(d["parents"], many)
    table = shift(np.where(np.arange(9) < -(-d["ctx"][:, None] // 16), d["table"], -1))
    # pages of the list in the order in which the requests take them
    first = np.concatenate([d["free"][:d["first"]] + i * d["blocks"] for i in range(many)])
    free = np.concatenate([first] + [d["free"][d["first"]:d["head"]] + i * d["blocks"] for i in range(many)]
                          + [d["free"][d["head"]:] + i * d["blocks"] for i in range(many)])
    k, v = _caches(5, None, many * d["blocks"], 1, 16, 8)
    lens, ids, t = _i32(ctx), _i32(free), _i32(table)
    plan = dgt.dgt_page_plan(lens, _i32(new), ids, _i32([len(first)]), t, 16, many * d["blocks"], int(new.sum()),
                             parents=_i32(parents))
    assert plan.counts.tolist() == [int(new.sum()), many * d["head"], 0]
    assert np.array_equal(t.cpu().numpy(), shift(d["table"]))
    kd, vd = k.cuda(), v.cuda()
    counts = dgt.dgt_page_keep(_i32(kept * many), lens, plan.cu, plan.slots, ids, plan.counts[1:2], t, kd, vd)
    assert lens.tolist() == (ctx + np.array(kept * many)).tolist()
    held_or_free(dict(d, blocks=many * d["blocks"]), t.tolist(), lens.tolist(), ids.tolist(), int(counts[0]))
    assert torch.equal(_bits(kd), _bits(k)) and torch.equal(_bits(vd), _bits(v))


def test_keep_ends_a_path_at_a_row_without_a_slot():
    """Rows past the mask, behind a bad link, and places without a slot; in the first 16 rows of a path, behind
    them, and far behind, with requests before and after that keep all."""
    from tests.test_oracle_step import odd_step
    d = odd_step()
    path = np.full(190, -1)
    path[:4], path[100:104], path[140:142], path[170:173] = [0, 60, 63, 64], [0, 5, 11, 12], [0, 1], [0, 3, 4]
    for in_place in (True, False):
        _keep(d, path, [4, 4, 2, 3], 2, 2, 40, in_place=in_place)
        _keep(d, None, [100, 40, 30, 20], 2, 2, 40, in_place=in_place)
        _keep(d, np.concatenate([np.arange(n) for n in d["new"]]), [100, 40, 30, 20], 1, 1, 8, in_place=in_place)
    rng = np.random.default_rng(8)
    new = [3000, 20, 0, 700, 40, 1, 2000] + [12] * 300
    d = _step(23, rng.integers(0, 50, len(new)), new, 16)
    start = np.concatenate([[0], np.cumsum(new)])
    for b, row in ((0, 2900), (1, 17), (3, 15), (4, 16), (6, 1999), (8, 3), (200, 11)):
        d["slots"][start[b] + row] = -1
    kept = np.array(new) - rng.integers(0, 2, len(new))
    _keep(d, None, kept, None, 1, 8)
    # upward paths that leave out a row in three
    path = np.full(sum(new), -1)
    for b, n in enumerate(new):
        way = np.array([i for i in range(n) if i % 3 != 1])
        path[start[b]:start[b] + len(way)] = way
        kept[b] = len(way)
    _keep(d, path, kept, 2, 1, 8)
    _keep(d, path, kept, None, 1, 24, "float16", in_place=False)
