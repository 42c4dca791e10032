"""Attention over the paged cache against the 64-bit oracle.

Tolerance: with u the unit roundoff of the 16-bit type (2^-8 for bf16, 2^-11 for
fp16), |out - ref| <= u |ref| for the result's own rounding, plus u A for that of the
weights, A the weighted mean of |v|; 4e-4 A covers the fp32 scores (128 products of
values of a few units: below 1e-4 in the exponent), exponentials and sums.  In fp16
weights below 2^-14 round to a multiple of 2^-24: at most 2^-25 * keys * max |v| more."""

import numpy as np
import pytest

import decode_gemm_tile_amd as dgt
from oracle import serving

pytestmark = pytest.mark.gpu


def _i32(a):
    import torch
    return torch.from_numpy(np.ascontiguousarray(np.asarray(a, np.int32))).to("cuda")


def _make(seed, ctx, new, heads, kv_heads, dim, block, dtype="bfloat16", words=None, extra=2, spread=1.0):
    """Requests with random trees (words given) or chains; pages not in use hold NaN."""
    import torch
    g = torch.Generator().manual_seed(seed)
    rng = np.random.default_rng(seed)
    dtype = getattr(torch, dtype)
    pages = [-(-(c + n) // block) for c, n in zip(ctx, new)]
    blocks, width = sum(pages) + extra, max(pages) + 1
    ids, at = rng.permutation(blocks), 0
    table = np.full((len(ctx), width), -1)
    kc = torch.full((blocks, kv_heads, block, dim), float("nan"))
    vc = torch.full((blocks, kv_heads, dim, block), float("nan"))
    for b, p in enumerate(pages):
        table[b, :p] = ids[at:at + p]
        at += p
        count = ctx[b] + new[b]
        for j in range(p):  # cells past the request's tokens stay NaN
            live = min(block, count - j * block)
            kc[table[b, j], :, :live] = torch.randn((kv_heads, live, dim), generator=g) * spread
            vc[table[b, j], :, :, :live] = torch.randn((kv_heads, dim, live), generator=g)
    q = torch.randn((sum(new), heads, dim), generator=g) * spread
    seen = []
    for n in new:
        if words is None:
            seen.append(np.tril(np.ones((n, n), bool)))
        else:
            s = serving.ancestors([int(rng.integers(-1, i)) for i in range(n)]) if n else np.zeros((0, 0), bool)
            s[:, 64 * words:] = False
            seen.append(s)
    return dict(q=q.to(dtype), kc=kc.to(dtype), vc=vc.to(dtype), table=table, ctx=list(ctx), new=list(new),
                cu=np.concatenate([[0], np.cumsum(new)]), seen=seen, words=words, block=block)


def _mask(d):
    import torch
    if d["words"] is None:
        return None
    rows = [serving.pack_mask(s, d["words"]) for s in d["seen"]]
    return torch.from_numpy(np.concatenate(rows).view(np.int64)).cuda()


def _run(d, **kw):
    import torch
    out = dgt.dgt_tree_attention(d["q"].cuda(), d["kc"].cuda(), d["vc"].cuda(), _i32(d["table"]), _i32(d["ctx"]),
                                 _i32(d["cu"]), mask=_mask(d), **kw)
    torch.cuda.synchronize()
    return out


def _check(d, out, scale=None, requests=None):
    import torch
    u, low = (2.0 ** -8, 0.0) if d["q"].dtype is torch.bfloat16 else (2.0 ** -11, 2.0 ** -25)
    scale = d["q"].shape[2] ** -0.5 if scale is None else scale
    q, kc, vc = (d[x].double().numpy() for x in ("q", "kc", "vc"))
    got = out.double().cpu().numpy()
    for b, (c, n) in enumerate(zip(d["ctx"], d["new"])):
        if requests is not None and b not in requests:
            continue
        s, e = d["cu"][b], d["cu"][b + 1]
        keys, values = serving.gather(kc, vc, d["table"][b], c + n)
        ref, size = serving.tree_attention(q[s:e], keys, values, c, d["seen"][b], scale)
        top = np.abs(values[np.isfinite(values)]).max() if values.size else 0.0
        tol = u * np.abs(ref) + (u + 4e-4) * size + low * (c + n) * top
        err = np.abs(got[s:e] - ref)
        assert (err <= tol).all(), (b, float(np.nanmax(err - tol)), np.isnan(got[s:e]).any())


SHAPES = [  # ctx, new, heads, kv_heads, dim, block
    ([0], [1], 1, 1, 64, 16),
    ([1], [1], 4, 1, 128, 16),
    ([31], [1], 8, 2, 128, 16),
    ([32], [1], 8, 8, 64, 32),
    ([127, 128, 129], [1, 1, 1], 4, 2, 128, 16),
    ([1000], [1], 8, 2, 128, 16),
    ([0, 500, 3, 77], [0, 5, 0, 1], 6, 2, 64, 8),
    ([300, 0, 41], [7, 9, 30], 8, 2, 128, 16),
    ([700, 15], [40, 61], 16, 2, 128, 64),
    ([511, 90], [13, 64], 4, 4, 80, 16),
    ([100, 260], [3, 20], 6, 2, 72, 128),
    ([65, 200], [4, 33], 4, 2, 256, 16),
    ([30, 0], [11, 2], 4, 1, 200, 32),
    ([5, 19], [6, 1], 3, 3, 8, 8),
    ([2500], [2], 32, 2, 128, 1024),
    ([60] * 40, [2] * 40, 4, 1, 64, 16),
    ([9] * 300, [1] * 300, 2, 1, 64, 16),
    # few rows on the average, many in one request; with a long context too
    ([300] + [20] * 30, [40] + [1] * 30, 4, 2, 128, 16),
    ([30000] + [5] * 30, [40] + [1] * 30, 2, 1, 64, 64),
    # narrower heads than the kernels are made for, at every number of rows
    ([77, 1200], [1, 2], 4, 2, 104, 16),
    ([50, 300], [20, 3], 4, 2, 40, 16),
    ([120], [40], 4, 1, 96, 16),
    ([100, 7], [64, 50], 4, 2, 48, 32),
]


@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
@pytest.mark.parametrize("words", [None, 1], ids=["chain", "tree"])
@pytest.mark.parametrize("i", range(len(SHAPES)))
def test_attention_against_oracle(i, words, dtype):
    d = _make(i + 1, *SHAPES[i], dtype=dtype, words=words)
    _check(d, _run(d))


@pytest.mark.parametrize("new,words", [([70, 130], 3), ([65], 2), ([128, 5], 2), ([200], 2), ([129], 1)])
def test_trees_wider_than_a_word(new, words):
    """More drafted tokens than 64; where the mask has too few words, bits past them are unset."""
    d = _make(50 + len(new), [45, 200][:len(new)], new, 4, 2, 64, 16, words=words)
    _check(d, _run(d))


@pytest.mark.parametrize("offset", range(0, 40, 3))
def test_drafted_keys_at_every_place_of_a_tile(offset):
    """ctx from 190 to 229: the drafted keys begin anywhere within 8 and 32 keys."""
    d = _make(80 + offset, [190 + offset, 64 + offset], [60, 25], 4, 2, 64, 16, words=1)
    _check(d, _run(d))


@pytest.mark.parametrize("ctx,new,heads,kv,dtype", [([0], [1000], 4, 2, "bfloat16"), ([77, 0], [300, 1100], 4, 1, "bfloat16"),
                                                    ([1500, 9, 0], [513, 1, 2], 2, 2, "float16")])
def test_prompts(ctx, new, heads, kv, dtype):
    """Chains of many new tokens, with and without cached ones, split between workgroups."""
    d = _make(len(new) + 200, ctx, new, heads, kv, 64, 16, dtype=dtype)
    _check(d, _run(d))


def _device_reference(q, kc, vc, pages, ctx, n, see, scale):
    """float64 on the device for one request, head by head (the oracle takes minutes at this size).
    q [n, heads, dim]; see [n, n] over the new tokens.  Returns (out, weighted mean of |v|)."""
    import torch
    heads, dim = q.shape[1:]
    group = heads // kc.shape[1]
    out, size = (torch.empty(q.shape, dtype=torch.float64, device="cuda") for _ in range(2))
    seen = torch.cat([torch.ones((n, ctx), dtype=torch.bool), torch.from_numpy(see)], 1).cuda()
    for g in range(kc.shape[1]):
        keys = kc[pages, g].reshape(-1, dim)[:ctx + n].double().t().contiguous()
        values = vc[pages, g].transpose(1, 2).reshape(-1, dim)[:ctx + n].double().contiguous()
        for h in range(g * group, (g + 1) * group):
            z = torch.mm(q[:, h].double(), keys) * scale
            w = torch.softmax(z.masked_fill(~seen, -float("inf")), 1)
            out[:, h], size[:, h] = torch.mm(w, values), torch.mm(w, values.abs())
    return out, size


@pytest.mark.parametrize("new", [5, 40])
def test_runs_of_more_pages_than_fit_in_lds(new):
    """Small pages and so many keys that one workgroup's run of them spans more than 1024 pages:
    8 requests of 80000 keys, 8 key heads.  Requests share their pages, as a common prefix would."""
    import torch
    heads, kv, dim, block, requests = 16, 8, 64, 8, 8
    ctx = [80000 - 999 * b for b in range(requests)]
    # units of 128 keys, dealt to 512 workgroups (one tile of rows); pages of 8 keys
    tiles = -(-new * heads // kv // 128)
    assert sum(c // 128 for c in ctx) * kv * tiles // 512 * (128 // block) > 1024
    g = torch.Generator(device="cuda").manual_seed(3)
    blocks = -(-(max(ctx) + new) // block)
    randn = lambda *s: torch.randn(s, generator=g, device="cuda").to(torch.bfloat16)
    kc, vc, q = randn(blocks, kv, block, dim), randn(blocks, kv, dim, block), randn(requests * new, heads, dim)
    pages = torch.randperm(blocks, generator=g, device="cuda")
    see = serving.ancestors([int(i) for i in np.random.default_rng(new).integers(-1, np.arange(new))])
    mask = torch.from_numpy(np.tile(serving.pack_mask(see, 1), (requests, 1)).view(np.int64)).cuda()
    out = dgt.dgt_tree_attention(q, kc, vc, pages.int().repeat(requests, 1).contiguous(), _i32(ctx),
                                 _i32(np.arange(requests + 1) * new), mask=mask)
    u = 2.0 ** -8
    for b, c in enumerate(ctx):
        rows = slice(b * new, (b + 1) * new)
        ref, size = _device_reference(q[rows], kc, vc, pages, c, new, see, dim ** -0.5)
        assert ((out[rows].double() - ref).abs() <= u * ref.abs() + (u + 4e-4) * size).all(), b


def test_sharp_softmax():
    """Scores of some hundreds: all weight on a few keys, maxima that move between tiles."""
    d = _make(90, [900, 333], [3, 20], 8, 2, 128, 16, words=1, spread=6.0)
    out = _run(d)
    # the bound's 4e-4 is for scores of a few units; at |s| ~ 500 fp32 scores are off by up to
    # 128 * 2^-24 * 128 * 36 / sqrt(128) ~ 3e-3, which moves the weights by as much
    u = 2.0 ** -8
    q, kc, vc = (d[x].double().numpy() for x in ("q", "kc", "vc"))
    for b in range(2):
        keys, values = serving.gather(kc, vc, d["table"][b], d["ctx"][b] + d["new"][b])
        s, e = d["cu"][b], d["cu"][b + 1]
        ref, size = serving.tree_attention(q[s:e], keys, values, d["ctx"][b], d["seen"][b], 128 ** -0.5)
        err = np.abs(out[s:e].double().cpu().numpy() - ref)
        assert (err <= u * np.abs(ref) + (u + 6e-3) * size).all()


def test_rows_that_see_nothing_are_zero():
    import torch
    d = _make(91, [0, 0, 40], [5, 33, 3], 8, 2, 128, 16, words=1)
    d["seen"][0][2] = False
    d["seen"][1][:] = False
    d["seen"][2][:] = False
    out = _run(d)
    assert (out[2] == 0).all() and (out[5:38] == 0).all()
    _check(d, out)
    # an empty mask on the first new token, nothing cached, alone
    d = _make(92, [0], [1], 2, 1, 64, 16, words=1)
    d["seen"][0][:] = False
    assert (_run(d) == 0).all()


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf"), 3e38])
@pytest.mark.parametrize("what", ["k", "v", "both"])
def test_unseen_keys_do_not_touch_a_row(bad, what):
    """A drafted key that a row does not see may hold anything; rows that see it get it."""
    import torch
    d = _make(93, [70, 10], [9, 20], 8, 2, 128, 16, words=1)
    clean = _run(d)
    for b, j in ((0, 4), (1, 0), (1, 13)):
        p = d["ctx"][b] + j
        page, cell = d["table"][b][p // 16], p % 16
        if what != "v":
            d["kc"][page, :, cell] = bad
        if what != "k":
            d["vc"][page, :, :, cell] = bad
        d["seen"][b][:, j] &= np.arange(len(d["seen"][b])) == j
    seen_bad = np.zeros(29, bool)
    seen_bad[[4, 9, 9 + 13]] = True
    base = {**d, "kc": torch.nan_to_num(d["kc"], nan=0.0, posinf=0.0, neginf=0.0).clamp(-9, 9),
            "vc": torch.nan_to_num(d["vc"], nan=0.0, posinf=0.0, neginf=0.0).clamp(-9, 9)}
    out, ref = _run(d), _run(base)
    assert torch.isfinite(out[~seen_bad]).all()
    # rows without the bad keys: the same as with harmless values in their place, within rounding
    # (a tile with values that are not finite is summed key by key)
    a, b = out[~seen_bad].float(), ref[~seen_bad].float()
    assert (a - b).abs().max() <= 4 * 2.0 ** -8 * b.abs().max()
    if what != "k" and not np.isfinite(bad):
        assert not torch.isfinite(out[seen_bad]).any()


def test_values_out_of_use_are_not_read_into_rows():
    """Cells past the tokens and pages past the table hold NaN in every case above; here the
    cells hold infinities and the table names a page outside the pool for an unused column."""
    import torch
    d = _make(94, [33, 8], [2, 1], 4, 2, 64, 16)
    d["kc"], d["vc"] = (torch.where(d[x].isnan(), torch.tensor(float("-inf"), dtype=d[x].dtype), d[x]) for x in ("kc", "vc"))
    d["table"][0, -1], d["table"][1, -1] = 2 ** 31 - 1, -7
    _check(d, _run(d))


def test_missing_pages_count_as_absent():
    """Keys on pages outside the pool are left out, as if the request did not have them."""
    import torch
    d = _make(95, [64], [1], 4, 2, 64, 16)
    full = _run(d)
    keep = [0, 1, 3, 4]
    part = dict(d, ctx=[48], table=d["table"][:, keep])
    hole = dict(d, table=d["table"].copy())
    hole["table"][0, 2] = 12345
    got = _run(hole)
    _check(part, got)
    assert not torch.equal(got, full)


@pytest.mark.parametrize("new", [1, 6, 40])
def test_equal_scores_give_the_mean_of_the_seen(new):
    """q = 0: exact weights, so the mean of what is seen, rounded once; a key too many or too
    few would move it by 1 / count."""
    d = _make(96 + new, [200], [new], 4, 2, 64, 16, words=1)
    d["q"].zero_()
    vals = d["vc"].float()
    d["vc"] = vals.nan_to_num(0.0).round().clamp(-2, 2).to(d["vc"].dtype)
    out = _run(d).double().cpu().numpy()
    _, values = serving.gather(d["kc"].double().numpy(), d["vc"].double().numpy(), d["table"][0], 200 + new)
    for i in range(new):
        see = np.concatenate([np.ones(200, bool), d["seen"][0][i]])
        for h in range(4):
            want = values[see, h // 2].mean(0)
            assert (np.abs(out[i, h] - want) <= 2.0 ** -8 * np.abs(want) + 1e-6).all()


def test_strides_of_queries_and_outputs():
    """q as a part of wider rows, out as a transposed part; what lies beside out stays."""
    import torch
    d = _make(97, [100, 7], [3, 12], 8, 2, 64, 16, words=1)
    plain = _run(d)
    wide = torch.full((15, 12, 72), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[:, 2:10, 8:72] = d["q"].cuda()
    room = torch.full((8, 15, 66), 5.0, dtype=torch.bfloat16, device="cuda")
    args = (d["kc"].cuda(), d["vc"].cuda(), _i32(d["table"]), _i32(d["ctx"]), _i32(d["cu"]))
    out = dgt.dgt_tree_attention(wide[:, 2:10, 8:72], *args, mask=_mask(d), out=room.transpose(0, 1)[:, :, 2:])
    assert torch.equal(out, plain)
    assert (room[:, :, :2] == 5).all()
    with pytest.raises(dgt.DgtError):  # rows that are not 16-byte aligned
        dgt.dgt_tree_attention(wide[:, 2:10, 1:65], *args, mask=_mask(d))


def test_single_rows_and_heads_of_any_stride():
    """The stride of a dimension of size one means nothing."""
    import torch
    for d in (_make(126, [50], [1], 4, 2, 64, 16), _make(127, [50], [3], 1, 1, 64, 16), _make(128, [9], [1], 1, 1, 64, 16)):
        q = d["q"].cuda()
        plain = _run(d)
        _check(d, plain)
        odd = tuple(13 if n == 1 else s for n, s in zip(q.shape[:2], q.stride())) + (1,)
        args = (d["kc"].cuda(), d["vc"].cuda(), _i32(d["table"]), _i32(d["ctx"]), _i32(d["cu"]))
        out = torch.empty_like(q).as_strided(q.shape, odd)
        assert torch.equal(dgt.dgt_tree_attention(q.as_strided(q.shape, odd), *args, out=out), plain)


def test_rows_past_the_requests_are_not_written():
    import torch
    d = _make(98, [20], [3], 4, 2, 64, 16)
    q = torch.cat([d["q"], torch.full((5, 4, 64), float("nan"), dtype=torch.bfloat16)]).cuda()
    out = torch.full_like(q, 3.0)
    dgt.dgt_tree_attention(q, d["kc"].cuda(), d["vc"].cuda(), _i32(d["table"]), _i32(d["ctx"]), _i32(d["cu"]), out=out)
    _check(d, out[:3])
    assert (out[3:] == 3).all()


@pytest.mark.parametrize("ctx,new,heads,kv", [([4000], [1], 8, 1), ([5000, 10], [9, 2], 16, 2), ([3000], [40], 16, 2)])
def test_long_contexts_repeat_bit_for_bit(ctx, new, heads, kv):
    """Many workgroups share a row's keys; one workspace serves calls of other sizes in
    between, and the result does not depend on who comes last."""
    import torch
    d = _make(99, ctx, new, heads, kv, 128, 16, words=1)
    small = _make(100, [50], [2], 4, 2, 128, 16)
    big = max(dgt.dgt_tree_attention_workspace(x["q"].shape, x["kc"].shape[1], len(x["ctx"])) for x in (d, small))
    ws = dgt.alloc_workspace(big)
    first = _run(d, ws=ws)
    _check(d, first)
    for _ in range(3):
        _check(small, _run(small, ws=ws))
        assert torch.equal(_run(d, ws=ws), first)


def test_one_workspace_for_every_kind_of_call():
    """Calls with few and with many rows, each with as many parts as there can be, take turns
    on one workspace: the parts of one never lie where another counts."""
    import torch
    few = _make(120, [50000], [1], 8, 8, 64, 64, extra=0)
    many = _make(121, [9000, 6000], [40, 30], 8, 2, 64, 64, words=1, extra=0)
    some = _make(122, [9000], [9], 8, 2, 128, 64, words=1, extra=0)
    cases = (few, many, some)
    own = [_run(d) for d in cases]  # each on a workspace of its own
    ws = dgt.alloc_workspace(max(dgt.dgt_tree_attention_workspace(d["q"].shape, d["kc"].shape[1], len(d["ctx"]))
                                 for d in cases))
    for i in (0, 1, 0, 2, 0, 1, 2, 0):
        assert torch.equal(_run(cases[i], ws=ws), own[i]), i


def test_only_the_counters_are_cleared(monkeypatch):
    """The parts of a workspace may hold anything before its first use, and a call that makes
    its own clears no more of it than the counters."""
    import torch
    cases = [_make(124, [3000], [1], 8, 2, 128, 16), _make(125, [3000, 900], [40, 9], 16, 2, 128, 16, words=1)]
    for d in cases:
        nbytes = dgt.dgt_tree_attention_workspace(d["q"].shape, 2, len(d["ctx"]))
        assert nbytes > 100 * dgt.DGT_TREE_ATTENTION_ZEROED
        ws = torch.full((nbytes,), 0xFF, dtype=torch.uint8, device="cuda")  # NaN in fp32
        ws[:dgt.DGT_TREE_ATTENTION_ZEROED] = 0
        want = _run(d, ws=ws)
        _check(d, want)
        made, cleared = torch.zeros, []
        monkeypatch.setattr(torch, "zeros", lambda *a, **kw: cleared.append(made(*a, **kw)) or cleared[-1])
        assert torch.equal(_run(d), want)
        monkeypatch.undo()
        assert all(t.nbytes <= dgt.DGT_TREE_ATTENTION_ZEROED for t in cleared)


def test_scale_is_taken():
    d = _make(101, [150], [4], 4, 2, 64, 16)
    for scale in (1e-3, 0.3):
        _check(d, _run(d, scale=scale), scale=scale)


def test_garbage_offsets_and_lengths_stay_inside():
    """Device data that no plan makes: the call returns, and a sound one after it is right."""
    import torch
    d = _make(102, [40, 50], [3, 4], 4, 2, 64, 16, words=1)
    q, kc, vc, table, mask = d["q"].cuda(), d["kc"].cuda(), d["vc"].cuda(), _i32(d["table"]), _mask(d)
    ws = dgt.alloc_workspace(dgt.dgt_tree_attention_workspace(q.shape, 2, 2))
    for ctx, cu in (([2 ** 31 - 1, -5], [0, 3, 7]), ([40, 50], [0, 2 ** 31 - 1, 7]), ([40, 50], [5, 2, 99]),
                    ([40, 50], [-9, -1, 7]), ([0, 0], [0, 0, 0])):
        guard = torch.full((9, 4, 64), 3.0, dtype=torch.bfloat16, device="cuda")
        dgt.dgt_tree_attention(q, kc, vc, table, _i32(ctx), _i32(cu), mask=mask, out=guard[1:8], ws=ws)
        torch.cuda.synchronize()
        assert (guard[0] == 3).all() and (guard[8] == 3).all()
    _check(d, _run(d, ws=ws))


def test_offsets_that_name_rows_again_and_again():
    """Offsets that go up and down over 1024 requests with full tables: 8.6e9 units of work, more
    than 32 bits hold.  Nothing is written; a sound call on the same workspace after it is right."""
    import torch
    requests, tokens, heads, kv, dim, block, width = 1024, 65536, 32, 8, 8, 1024, 128
    # units: 512 requests of 65536 * 4 rows in tiles of 128, tables of 1024 times 128 keys, 8 heads
    assert 512 * (tokens * 4 // 128) * (width * block // 128) * kv >= 2 ** 33
    q = torch.zeros((tokens, heads, dim), dtype=torch.bfloat16, device="cuda")
    kc = torch.zeros((2, kv, block, dim), dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros((2, kv, dim, block), dtype=torch.bfloat16, device="cuda")
    table, ctx = _i32(np.zeros((requests, width))), _i32([2 ** 31 - 1] * requests)
    cu = np.zeros(requests + 1)
    cu[1::2] = tokens
    ws = dgt.alloc_workspace(dgt.dgt_tree_attention_workspace(q.shape, kv, requests))
    out = torch.full_like(q, 3.0)
    dgt.dgt_tree_attention(q, kc, vc, table, ctx, _i32(cu), out=out, ws=ws)
    torch.cuda.synchronize()
    assert (out == 3).all()
    d = _make(123, [700, 40], [40, 30], 8, 2, 64, 16, words=1)
    _check(d, _run(d, ws=ws))


def test_pool_past_32_bit_offsets():
    """Pages at both ends of a pool of more than 2^32 elements."""
    import torch
    d = _make(103, [300], [5], 8, 8, 128, 128, extra=0)
    blocks = 33000
    kc = torch.empty((blocks, 8, 128, 128), dtype=torch.bfloat16, device="cuda")
    vc = torch.empty((blocks, 8, 128, 128), dtype=torch.bfloat16, device="cuda")
    assert kc.numel() > 2 ** 32
    where = [blocks - 1, 3, blocks - 2]
    for j, page in enumerate(d["table"][0, :3]):
        kc[where[j]], vc[where[j]] = d["kc"][page].cuda(), d["vc"][page].cuda()
    out = dgt.dgt_tree_attention(d["q"].cuda(), kc, vc, _i32([where]), _i32([300]), _i32([0, 5]))
    _check(d, out)


def test_on_another_stream():
    import torch
    d = _make(104, [2000, 30], [2, 11], 8, 2, 128, 16, words=1)
    first = _run(d)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    assert torch.equal(_run(d, stream=s), first)
    with torch.cuda.stream(s):
        again = _run(d)
    assert torch.equal(again, first)


def test_in_a_graph():
    """Captured once; replays follow the lengths, tables and queries then in the tensors."""
    import torch
    cases = [_make(105 + i, c, n, 8, 2, 128, 16, words=1) for i, (c, n) in
             enumerate((([900, 40], [3, 8]), ([10, 700], [8, 3]), ([33, 2], [4, 7])))]
    blocks = max(c["kc"].shape[0] for c in cases)
    width = max(c["table"].shape[1] for c in cases)
    q = torch.empty((11, 8, 128), dtype=torch.bfloat16, device="cuda")
    kc = torch.empty((blocks, 2, 16, 128), dtype=torch.bfloat16, device="cuda")
    vc = torch.empty((blocks, 2, 128, 16), dtype=torch.bfloat16, device="cuda")
    table, ctx, cu = _i32(np.zeros((2, width))), _i32([0, 0]), _i32([0, 0, 0])
    mask, out = torch.zeros((11, 1), dtype=torch.int64, device="cuda"), torch.empty_like(q)
    ws = dgt.alloc_workspace(dgt.dgt_tree_attention_workspace(q.shape, 2, 2))

    def fill(c):
        q.copy_(c["q"]), kc[:len(c["kc"])].copy_(c["kc"]), vc[:len(c["vc"])].copy_(c["vc"])
        table[:, :c["table"].shape[1]].copy_(_i32(c["table"]))
        ctx.copy_(_i32(c["ctx"])), cu.copy_(_i32(c["cu"])), mask.copy_(_mask(c))

    def call():
        dgt.dgt_tree_attention(q, kc, vc, table, ctx, cu, mask=mask, out=out, ws=ws)

    fill(cases[0])
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for c in cases + cases[:1]:
        fill(c)
        out.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        _check(c, out)
        replayed = out.clone()
        call()
        torch.cuda.synchronize()
        assert torch.equal(out, replayed)
