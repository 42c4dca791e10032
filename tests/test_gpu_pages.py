"""Page plan and cache store against the plain forms: whole numbers equal, stored
values bit for bit."""

import numpy as np
import pytest

import decode_gemm_tile_amd as dgt
from oracle import serving

pytestmark = pytest.mark.gpu


def _dev(a, dtype=np.int32):
    import torch
    return torch.from_numpy(np.ascontiguousarray(np.asarray(a, dtype))).to("cuda")


def _plan_case(seed, requests, ctx, new, block, width=None, slack=5, tree=False, words=1, head=2, tokens=None):
    """Random lengths up to ctx and new, with zeros and whole pages among them."""
    rng = np.random.default_rng(seed)
    c = rng.integers(0, ctx + 1, requests)
    n = rng.integers(0, new + 1, requests)
    c[::5] = c[::5] // block * block
    n[3::7] = 0
    have = -(-c // block)
    need = -(-(c + n) // block) - have
    width = int((-(-(c + n) // block)).max()) if width is None else width
    total = int(have.sum()) + int(need.sum()) + slack + head
    ids = rng.permutation(total)
    table = np.full((requests, max(width, 0)), -1)
    at = 0
    for b in range(requests):
        table[b, :have[b]] = ids[at:at + have[b]][:width]
        at += have[b]
    free = ids[at:]
    parents = None
    if tree:
        parents = np.concatenate([[rng.integers(-1, i) for i in range(k)] for k in n] + [[]]).astype(np.int64)
    tokens = int(n.sum()) if tokens is None else tokens
    if tree and tokens > len(parents):
        parents = np.concatenate([parents, np.zeros(tokens - len(parents), np.int64)])
    return dict(ctx=c, new=n, free=free, head=head, table=table, block=block, blocks=total, tokens=tokens,
                parents=None if parents is None else parents[:tokens], words=words if tree else 0)


def _check_plan(case, out=None, stream=None):
    import torch
    table = _dev(case["table"])
    p = dgt.dgt_page_plan(_dev(case["ctx"]), _dev(case["new"]), _dev(case["free"]), _dev([case["head"]]), table,
                          case["block"], case["blocks"], case["tokens"],
                          parents=None if case["parents"] is None else _dev(case["parents"]),
                          mask_words=case["words"], out=out, stream=stream)
    torch.cuda.synchronize()
    want = serving.page_plan(case["ctx"], case["new"], case["free"], case["head"], case["table"], case["block"],
                             case["blocks"], case["tokens"], case["parents"], case["words"])
    for name, got, ref in zip(("table", "cu", "slots", "positions", "mask", "counts"),
                              (table, p.cu, p.slots, p.positions, p.mask, p.counts), want):
        if ref is None:
            assert got is None
            continue
        got = got.cpu().numpy()
        got = got.view(np.uint64) if name == "mask" else got.astype(np.int64)
        assert np.array_equal(got, ref), name
    return p, want


@pytest.mark.parametrize("block", [8, 16, 64, 1024])
@pytest.mark.parametrize("requests,ctx,new", [(1, 0, 1), (1, 50, 1), (5, 100, 3), (65, 3000, 40), (300, 500, 9)])
def test_plan_of_chains(block, requests, ctx, new):
    _check_plan(_plan_case(requests + block, requests, ctx, new, block))


@pytest.mark.parametrize("requests,new,words", [(1, 1, 1), (3, 64, 1), (40, 13, 1), (7, 200, 4), (5, 130, 2), (4, 64, 3)])
def test_plan_of_trees(requests, new, words):
    """Trees of more nodes than the mask has bits are among them (5 requests of up to 130)."""
    _check_plan(_plan_case(17 * requests, requests, 700, new, 16, tree=True, words=words))


def test_plan_of_a_deep_chain_as_a_tree():
    n = 1000
    case = dict(ctx=[33], new=[n], free=np.arange(70), head=0, table=np.full((1, 70), 3), block=16, blocks=80,
                tokens=n, parents=np.arange(n) - 1, words=16)
    p, want = _check_plan(case)
    assert want[3][-1] == 33 + n - 1


@pytest.mark.parametrize("what", ["free list", "table", "rows"])
def test_plan_refuses_what_does_not_fit(what):
    case = _plan_case(5, 60, 400, 50, 16, slack=0, tree=True)
    if what == "free list":
        case["free"] = case["free"][:len(case["free"]) // 2]
    elif what == "table":
        case["table"] = np.ascontiguousarray(case["table"][:, :20])
    else:
        case["tokens"] = case["tokens"] // 2
        case["parents"] = case["parents"][:case["tokens"]]
    _, want = _check_plan(case)
    assert want[5][2] > 3


def test_plan_rows_past_the_requests_are_marked():
    case = _plan_case(6, 9, 100, 8, 16, tree=True)
    case["tokens"] += 300
    case["parents"] = np.concatenate([case["parents"], np.zeros(300, np.int64)])
    p, _ = _check_plan(case)
    assert (p.slots[-300:] == -1).all() and (p.positions[-300:] == -1).all() and (p.mask[-300:] == 0).all()


def test_plan_bad_parents_spoil_only_their_descendants():
    case = _plan_case(8, 12, 90, 30, 16, tree=True)
    case["parents"][::11] = 1000
    case["parents"][5::13] = -2
    case["parents"][7::17] = 2 ** 31 - 1
    _, want = _check_plan(case)
    assert (want[3] == -1).any() and (want[3] >= 0).any()


def test_plan_of_nothing():
    for requests, tokens in ((0, 0), (0, 5), (4, 0)):
        case = dict(ctx=[7] * requests, new=[0] * requests, free=np.zeros(0, np.int64), head=0,
                    table=np.zeros((requests, 3), np.int64), block=16, blocks=4, tokens=tokens, parents=None, words=0)
        _check_plan(case)


@pytest.mark.parametrize("requests", [4096, 4800, 5200, 5461, 8192])
def test_plan_of_many_requests(requests):
    """Up to the most there may be; around 5000 the sums' LDS passes what a plain launch has."""
    _check_plan(_plan_case(11, requests, 60, 3, 16))


def test_plan_of_garbage_lengths_stays_inside():
    """Lengths that are negative or near 2^31, a free list head past its end, page ids out
    of the pool: nothing but slots of -1 comes of them, and the sound requests are served."""
    case = dict(ctx=[5, -3, 2 ** 31 - 1, 9, 2 ** 31 - 9, 16], new=[1, 2, 3, 2 ** 31 - 1, 5, 1],
                free=np.array([6, 7, 8]), head=1, table=np.full((6, 4), 3), block=16, blocks=9, tokens=40,
                parents=None, words=0)
    case["table"][0, 0], case["table"][5, 1] = 77, -5
    import torch
    table = _dev(case["table"])
    p = dgt.dgt_page_plan(_dev(case["ctx"]), _dev(case["new"]), _dev(case["free"]), _dev([1]), table, 16, 9, 40)
    torch.cuda.synchronize()
    slots = p.slots.cpu().numpy()
    assert slots[0] == -1                       # its page id lies outside the pool
    assert slots[1:3].tolist() == [7 * 16, 7 * 16 + 1]
    assert (slots[3:] == -1).all()
    assert p.counts.cpu().tolist()[0] == 41 and (p.cu.cpu().numpy() <= 40).all()
    p = dgt.dgt_page_plan(_dev([0]), _dev([1]), _dev([6]), _dev([9]), _dev([[3]]), 16, 9, 1)
    assert p.slots.item() == -1 and p.counts.cpu().tolist() == [1, 9, 1]


def test_plan_steps_chain_through_the_head():
    """Three steps of one batch: each takes its pages where the last one stopped."""
    import torch
    rng = np.random.default_rng(3)
    requests, block = 20, 16
    ctx, table, head = np.zeros(requests, np.int64), np.full((requests, 12), -1), 0
    free = rng.permutation(300)
    d_table, d_head, out = _dev(table), _dev([0]), None
    for step in range(3):
        new = rng.integers(0, 50, requests)
        tokens = 50 * requests
        out = dgt.dgt_page_plan(_dev(ctx), _dev(new), _dev(free), d_head, d_table, block, 300, tokens, out=out)
        table, cu, slots, pos, _, counts = serving.page_plan(ctx, new, free, head, table, block, 300, tokens)
        torch.cuda.synchronize()
        assert np.array_equal(d_table.cpu().numpy(), table)
        assert np.array_equal(out.slots.cpu().numpy(), slots)
        d_head, head = out.counts[1:2].clone(), int(counts[1])
        assert d_head.item() == head
        ctx = ctx + new
    used = table[table >= 0]
    assert len(set(used.tolist())) == len(used) == head


def _chained_steps(requests, most, steps, tree, run):
    """Steps that read the list's head out of the counts that they write.  run(call) makes one
    pass: call(out) is the plan, out the PagePlan that all steps share."""
    import torch
    rng = np.random.default_rng(requests)
    block, tokens, words = 16, most * requests, -(-most // 64) if tree else 0
    width, blocks = -(-most * steps // block), requests * (-(-most * steps // block) + 1)
    free = rng.permutation(blocks)
    d_ctx, d_new, d_free, d_table = _dev([0] * requests), _dev([0] * requests), _dev(free), _dev(np.full((requests, width), -1))
    d_parents = _dev(np.zeros(tokens)) if tree else None
    out = dgt.PagePlan.empty(requests, tokens, words)
    out.counts.zero_()
    table, ctx, head = np.full((requests, width), -1), np.zeros(requests, np.int64), 0

    def call():
        dgt.dgt_page_plan(d_ctx, d_new, d_free, out.counts[1:2], d_table, block, blocks, tokens, parents=d_parents,
                          mask_words=words, out=out)
        d_ctx.add_(d_new)

    step = run(call)
    d_ctx.zero_(), out.counts.zero_(), d_table.fill_(-1)
    for _ in range(steps):
        new = rng.integers(0, most + 1, requests)
        parents = None
        if tree:
            parents = np.concatenate([[rng.integers(-1, i) for i in range(n)] for n in new] + [np.zeros(tokens)])[:tokens]
            d_parents.copy_(_dev(parents))
            parents = parents.astype(np.int64)
        d_new.copy_(_dev(new))
        step()
        torch.cuda.synchronize()
        table, cu, slots, pos, mask, counts = serving.page_plan(ctx, new, free, head, table, block, blocks, tokens,
                                                                parents, words)
        for got, ref in ((d_table, table), (out.cu, cu), (out.slots, slots), (out.positions, pos), (out.counts, counts)):
            assert np.array_equal(got.cpu().numpy(), ref)
        if tree:
            assert np.array_equal(out.mask.cpu().numpy().view(np.uint64), mask)
        ctx, head = ctx + new, int(counts[1])
    used = table[table >= 0]
    assert len(set(used.tolist())) == len(used) == head > 0


@pytest.mark.parametrize("requests,most,tree", [(5, 40, False), (8, 32, False), (9, 32, True), (900, 50, False), (500, 70, True)])
def test_plan_steps_chain_in_fixed_buffers(requests, most, tree):
    """The head is read where the step writes the next one: with one workgroup (up to 256 rows)
    and with up to 176."""
    _chained_steps(requests, most, 5, tree, lambda call: call)


def test_plan_steps_chain_in_a_graph():
    """A captured step in fixed buffers, replayed: each replay goes on where the last one stopped."""
    import torch

    def capture(call):
        call()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call()
        return graph.replay

    _chained_steps(300, 50, 5, True, capture)


def test_plan_on_another_stream():
    import torch
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    case = _plan_case(21, 50, 300, 20, 16, tree=True)
    with torch.cuda.stream(s):
        _check_plan(case)
    torch.cuda.synchronize()


# ---------------------------------------------------------------------- store
def _slots(rng, tokens, blocks, block, runs=True):
    """Distinct slots: runs of neighbours that start anywhere, some rows skipped."""
    if runs:
        out, taken = [], set()
        while len(out) < tokens:
            page, at = rng.integers(0, blocks), rng.integers(0, block)
            for cell in range(at, min(block, at + rng.integers(1, 30))):
                slot = page * block + cell
                if slot not in taken and len(out) < tokens:
                    taken.add(slot)
                    out.append(slot)
        out = np.array(out)
    else:
        out = rng.permutation(blocks * block)[:tokens]
    out[3::11] = -1
    out[4::19] = blocks * block
    return out


@pytest.mark.parametrize("source,cache", [("float32", "bfloat16"), ("float32", "float16"),
                                          ("bfloat16", "bfloat16"), ("float16", "float16")])
@pytest.mark.parametrize("tokens,heads,dim,block", [(1, 1, 64, 16), (3, 8, 128, 16), (67, 2, 80, 8), (200, 3, 72, 32),
                                                    (33, 1, 256, 64), (65, 5, 8, 128), (130, 2, 128, 1024)])
def test_store_is_bit_exact(source, cache, tokens, heads, dim, block):
    import torch
    _store_case(torch.Generator().manual_seed(tokens * dim), getattr(torch, source), getattr(torch, cache), tokens,
                heads, dim, block)


def _store_case(g, source, cache, tokens, heads, dim, block, runs=True, stream=None):
    import torch
    blocks = max(6, 3 * tokens // block)
    x = torch.randn((tokens, 3 * heads, dim), generator=g)
    x[0, 0, :4] = torch.tensor([float("inf"), -float("inf"), float("nan"), -0.0])
    x[-1, -1, -3:] = torch.tensor([1e38, 65519.0, 1e-41])
    x = x.to(source).cuda()
    k, v = x[:, heads:2 * heads], x[:, 2 * heads:]  # strided views of fused rows
    kc = torch.randn((blocks, heads, block, dim), generator=g).to(cache).cuda()
    vc = torch.randn((blocks, heads, dim, block), generator=g).to(cache).cuda()
    slots = _slots(np.random.default_rng(tokens), tokens, blocks, block, runs)
    kw, vw = kc.clone(), vc.clone()
    for t, s in enumerate(slots):
        if 0 <= s < blocks * block:
            kw[s // block, :, s % block] = k[t].to(cache)
            vw[s // block, :, :, s % block] = v[t].to(cache)
    dgt.dgt_kv_store(k, v, _dev(slots), kc, vc, stream=stream)
    torch.cuda.synchronize()
    # NaNs compare by being NaN, all else bit for bit
    for got, want in ((kc, kw), (vc, vw)):
        same = (got.view(torch.int16) == want.view(torch.int16)) | (got.isnan() & want.isnan())
        assert same.all()


def test_store_of_scattered_slots():
    import torch
    _store_case(torch.Generator().manual_seed(1), torch.float32, torch.bfloat16, 300, 2, 64, 16, runs=False)


def test_store_broadcast_rows_and_head_strides():
    """A row stride of zero (one row for all slots) and heads in another order of memory."""
    import torch
    g = torch.Generator().manual_seed(2)
    k = torch.randn((1, 4, 64), generator=g).cuda().expand(9, 4, 64)
    v = torch.randn((4, 9, 64), generator=g).cuda().transpose(0, 1)
    kc, vc = torch.zeros((3, 4, 16, 64), dtype=torch.float16, device="cuda"), \
        torch.zeros((3, 4, 64, 16), dtype=torch.float16, device="cuda")
    dgt.dgt_kv_store(k, v, _dev(np.arange(20, 29)), kc, vc)
    flat_k = kc.permute(0, 2, 1, 3).reshape(48, 4, 64)
    flat_v = vc.permute(0, 3, 1, 2).reshape(48, 4, 64)
    assert torch.equal(flat_k[20:29], k.half()) and torch.equal(flat_v[20:29], v.half())
    assert (flat_k[:20] == 0).all() and (flat_v[29:] == 0).all()


def test_store_past_32_bit_offsets():
    """A pool of more than 2^32 elements: slots at both ends land where they should."""
    import torch
    blocks, heads, block, dim = 33000, 8, 128, 128    # 4.3e9 elements a tensor
    kc = torch.empty((blocks, heads, block, dim), dtype=torch.bfloat16, device="cuda")
    vc = torch.empty((blocks, heads, dim, block), dtype=torch.bfloat16, device="cuda")
    assert kc.numel() > 2 ** 32
    slots = [0, 16400 * block + 5, blocks * block - 1, (blocks - 2) * block + 64]
    k = torch.randn((4, heads, dim), device="cuda")
    dgt.dgt_kv_store(k, -k, _dev(slots), kc, vc)
    for t, s in enumerate(slots):
        assert torch.equal(kc[s // block, :, s % block], k[t].bfloat16())
        assert torch.equal(vc[s // block, :, :, s % block], (-k[t]).bfloat16())
