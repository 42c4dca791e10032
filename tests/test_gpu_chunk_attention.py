"""Attention of chunks of new tokens against the 64-bit oracle, with the inputs, NaN cells and
tolerance of the tree attention's tests (the same roundings: weights to the 16-bit type, fp32 sums,
one rounding of the result)."""

import numpy as np
import pytest

import decode_gemm_tile_amd as dgt
from tests import test_gpu_tree_attention as tree
from tests.test_gpu_tree_attention import _i32

pytestmark = pytest.mark.gpu


def _run(d, **kw):
    import torch
    out = dgt.dgt_chunk_attention(d["q"].cuda(), d["kc"].cuda(), d["vc"].cuda(), _i32(d["table"]), _i32(d["ctx"]),
                                  _i32(d["cu"]), **kw)
    torch.cuda.synchronize()
    return out


SHAPES = [  # ctx, new, heads, kv_heads, dim, block
    ([0], [1], 1, 1, 64, 16),
    ([1], [1], 4, 1, 128, 16),
    ([63], [2], 8, 2, 128, 16),
    ([0], [64], 4, 1, 128, 16),
    ([0], [65], 4, 1, 128, 16),
    ([5], [129], 8, 2, 128, 16),
    ([0], [257], 2, 2, 64, 32),
    ([64, 127, 128], [1, 300, 63], 4, 2, 128, 64),
    ([0, 500, 3, 77], [0, 5, 0, 130], 6, 2, 64, 8),
    ([511, 90], [13, 200], 4, 4, 80, 16),
    ([100, 260], [31, 90], 6, 2, 72, 128),
    ([65, 200], [140, 33], 4, 2, 256, 16),
    ([30, 0], [11, 270], 4, 1, 200, 32),
    ([5, 19], [6, 40], 3, 3, 8, 8),
    ([2500], [20], 32, 2, 128, 1024),
    ([60] * 40, [2] * 40, 4, 1, 64, 16),
    ([20] * 30 + [9], [1] * 30 + [170], 10, 2, 128, 16),
    ([50, 300], [20, 100], 4, 2, 40, 16),
    # groups that leave rows of a tile over, and groups longer than a tile
    ([70], [90], 7, 1, 64, 16),
    ([40], [7], 300, 1, 64, 16),
    ([33], [5], 520, 2, 16, 16),
    ([33], [3], 131, 1, 256, 8),
]


@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
@pytest.mark.parametrize("i", range(len(SHAPES)))
def test_chunk_against_oracle(i, dtype):
    d = tree._make(i + 1, *SHAPES[i], dtype=dtype)
    tree._check(d, _run(d))


@pytest.mark.parametrize("offset", range(0, 70, 9))
def test_new_keys_at_every_place_of_a_tile(offset):
    d = tree._make(80 + offset, [190 + offset, offset], [60, 75], 4, 2, 64, 16)
    tree._check(d, _run(d))


LONG = [  # ctx, new, heads, kv_heads, dim, block, dtype: what is cut over its keys, and what is not
    ([9000], [5], 8, 2, 128, 16, "bfloat16"),
    ([20000], [100], 8, 1, 128, 64, "bfloat16"),
    ([100000], [1], 4, 1, 64, 32, "float16"),
    ([30000, 7, 0, 3000], [40, 900, 0, 1], 8, 2, 128, 16, "bfloat16"),
    ([0], [3000], 8, 2, 128, 16, "bfloat16"),
    ([1000], [2500], 4, 4, 128, 32, "float16"),
    ([7000, 100], [300, 700], 6, 2, 256, 16, "bfloat16"),
    ([5000] * 3, [120, 1, 60], 12, 4, 80, 16, "bfloat16"),
    ([3000] + [10] * 1500, [50] + [1] * 1500, 2, 1, 64, 16, "bfloat16"),
]


def _long(ctx, new, heads, kv_heads, dim, block, dtype, seed=0, spread=1.2):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    dtype = getattr(torch, dtype)
    pages = [-(-(c + n) // block) for c, n in zip(ctx, new)]
    ids, at = np.random.default_rng(seed).permutation(sum(pages) + 1), 0
    table = np.full((len(ctx), max(pages) + 1), -1)
    for b, p in enumerate(pages):
        table[b, :p] = ids[at:at + p]
        at += p
    made = lambda shape, s: (torch.randn(shape, generator=g, device="cuda") * s).to(dtype)
    return dict(q=made((sum(new), heads, dim), spread), kc=made((sum(pages) + 1, kv_heads, block, dim), spread),
                vc=made((sum(pages) + 1, kv_heads, dim, block), 1.0), table=_i32(table), ctx=ctx, new=new,
                cu=np.concatenate([[0], np.cumsum(new)]))


def _check_long(d, out):
    """The same definition and tolerance in float64 on the GPU, head by head."""
    import torch
    u, low = (2.0 ** -8, 0.0) if d["q"].dtype is torch.bfloat16 else (2.0 ** -11, 2.0 ** -25)
    kv, block, dim = d["kc"].shape[1], d["kc"].shape[2], d["kc"].shape[3]
    group = d["q"].shape[1] // kv
    for b, (c, n) in enumerate(zip(d["ctx"], d["new"])):
        if n == 0 or (len(d["ctx"]) > 100 and b % 97):
            continue
        s, e = int(d["cu"][b]), int(d["cu"][b + 1])
        ids = d["table"][b, :-(-(c + n) // block)].long()
        hidden = torch.ones((n, c + n), dtype=torch.bool, device="cuda").triu(c + 1)
        for h in range(d["q"].shape[1]):
            k = d["kc"][ids, h // group].reshape(-1, dim)[:c + n].double()
            v = d["vc"][ids, h // group].transpose(1, 2).reshape(-1, dim)[:c + n].double()
            z = (d["q"][s:e, h].double() @ k.t() * dim ** -0.5).masked_fill(hidden, float("-inf"))
            w = torch.softmax(z, 1)
            ref, size = w @ v, w @ v.abs()
            tol = u * ref.abs() + (u + 4e-4) * size + low * (c + n) * v.abs().max()
            err = (out[s:e, h].double() - ref).abs()
            assert bool((err <= tol).all()), (b, h, float((err - tol).max()))


@pytest.mark.parametrize("i", range(len(LONG)))
def test_long_chunks(i):
    import torch
    d = _long(*LONG[i], seed=i)
    run = lambda **kw: dgt.dgt_chunk_attention(d["q"], d["kc"], d["vc"], d["table"], _i32(d["ctx"]), _i32(d["cu"]), **kw)
    out = run()
    _check_long(d, out)
    ws = torch.full((dgt.dgt_chunk_attention_workspace(d["q"].shape, d["kc"].shape[1], len(d["ctx"])),), 255,
                    dtype=torch.uint8, device="cuda")
    for _ in range(2):  # bit for bit, whatever the workspace holds
        assert torch.equal(run(ws=ws), out)


def test_rows_behind_the_last_request_are_left():
    import torch
    d = tree._make(5, [40, 9], [30, 50], 4, 2, 64, 16)
    q = torch.cat([d["q"], torch.full((7, 4, 64), float("nan")).to(d["q"].dtype)]).cuda()
    out = torch.full_like(q, 3.0)
    dgt.dgt_chunk_attention(q, d["kc"].cuda(), d["vc"].cuda(), _i32(d["table"]), _i32(d["ctx"]), _i32(d["cu"]), out=out)
    assert bool((out[80:] == 3.0).all())
    tree._check(d, out[:80])


def test_strides_scale_and_streams():
    import torch
    d = tree._make(6, [100, 0], [33, 70], 6, 3, 80, 16)
    wide = torch.full((103, 20, 96), float("nan"), dtype=d["q"].dtype, device="cuda")
    q = wide[:, 3:9, 8:88]
    q.copy_(d["q"])
    out = torch.full((103, 9, 84), float("nan"), dtype=d["q"].dtype, device="cuda")[:, 2:8, 2:82]
    args = d["kc"].cuda(), d["vc"].cuda(), _i32(d["table"]), _i32(d["ctx"]), _i32(d["cu"])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = dgt.dgt_chunk_attention(q, *args, scale=0.31, out=out, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert got is out
    tree._check(d, out, scale=0.31)


def test_later_values_do_not_touch_earlier_rows():
    """A new token's value of infinity or NaN: rows before it are as without it; the others take it."""
    import torch
    d = tree._make(7, [70], [100], 4, 2, 128, 16)
    clean = _run(d)
    for at, bad in ((30, float("nan")), (64, float("inf"))):
        vc = d["vc"].clone()
        pos = 70 + at
        vc[d["table"][0][pos // 16], :, :, pos % 16] = bad
        out = _run(dict(d, vc=vc))
        # (key by key instead of in matrix products: the same sums within their tolerance)
        tree._check(dict(d, q=d["q"][:at], cu=[0, at], new=[at], seen=[np.tril(np.ones((at, at), bool))]), out[:at])
        assert not bool(torch.isfinite(out[at:]).any())
    assert bool(torch.isfinite(clean).all())


def test_missing_pages_are_not_seen():
    """Pages of -1 or out of range hold no keys; a request with none of its pages gives zeros."""
    import torch
    d = tree._make(8, [200, 40], [70, 10], 4, 2, 64, 16)
    table = np.array(d["table"])
    table[0, 5], table[1, :] = -1, 2 ** 30
    out = _run(dict(d, table=table))
    assert bool((out[70:] == 0).all())
    keep = np.r_[0:80, 96:270]
    q, kc, vc = (d[x].double().numpy() for x in ("q", "kc", "vc"))
    from oracle import serving
    keys, values = serving.gather(kc, vc, d["table"][0], 270)
    ref, size = serving.tree_attention(q[:70], keys[keep], values[keep], 184, np.tril(np.ones((70, 70), bool)), 64 ** -0.5)
    err = np.abs(out[:70].double().cpu().numpy() - ref)
    assert (err <= 2.0 ** -8 * np.abs(ref) + (2.0 ** -8 + 4e-4) * size).all()


def test_lengths_that_do_not_fit():
    """Negative contexts count as none; contexts past the table are cut to it; offsets that fall, or lie
    outside the rows, leave nothing written outside the rows."""
    import torch
    d = tree._make(9, [0], [60], 2, 1, 64, 16)
    tree._check(d, _run(dict(d, ctx=[-5])))
    args = [d["q"].cuda(), d["kc"].cuda(), d["vc"].cuda(), _i32(d["table"])]
    dgt.dgt_chunk_attention(*args, _i32([2 ** 31 - 1]), _i32([0, 60]))
    for cu in ([50, 10], [-7, 2 ** 31 - 1], [60, 60]):
        whole = torch.full((62, 2, 64), 5.0, dtype=d["q"].dtype, device="cuda")
        dgt.dgt_chunk_attention(*args, _i32([0]), _i32(cu), out=whole[1:61])
        assert bool((whole[0] == 5.0).all()) and bool((whole[61] == 5.0).all())
    two = torch.cat([args[3], args[3]])
    dgt.dgt_chunk_attention(args[0], args[1], args[2], torch.cat([two, two]), _i32([0] * 4), _i32([0, 60, 0, 60, 0]))
    torch.cuda.synchronize()


def test_captured_and_replayed():
    import torch
    d = _long([4000, 30], [60, 200], 8, 2, 128, 16, "bfloat16", seed=3)
    ctx, cu = _i32(d["ctx"]), _i32(d["cu"])
    ws = torch.zeros(dgt.dgt_chunk_attention_workspace(d["q"].shape, 2, 2), dtype=torch.uint8, device="cuda")
    out = torch.zeros_like(d["q"])
    run = lambda: dgt.dgt_chunk_attention(d["q"], d["kc"], d["vc"], d["table"], ctx, cu, out=out, ws=ws)
    run()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for c in (4000, 17, 2500):
        ctx[0] = c
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        _check_long(dict(d, ctx=[c, 30]), out)
        assert torch.equal(out, dgt.dgt_chunk_attention(d["q"], d["kc"], d["vc"], d["table"], ctx, cu))


def test_empty_calls():
    import torch
    d = tree._make(4, [3], [2], 2, 1, 64, 16)
    args = d["kc"].cuda(), d["vc"].cuda()
    none = torch.empty((0, 2, 64), dtype=d["q"].dtype, device="cuda")
    assert dgt.dgt_chunk_attention(none, *args, _i32(d["table"]), _i32([3]), _i32([0, 0])).numel() == 0


@pytest.mark.parametrize("dim,ctx,dtype", [(64, 0, "float16"), (80, 300, "bfloat16"), (128, 20000, "bfloat16"),
                                           (256, 500, "float16")])
def test_values_that_are_not_finite_reach_the_rows_that_see_them(dim, ctx, dtype):
    """Single elements of new tokens' values, in some tiles of the keys: their dimension becomes
    infinite or NaN in the rows from theirs on, all else is as with zeros in their places."""
    import torch
    d = _long([ctx], [200], 4, 2, dim, 16, dtype, seed=3)
    d["table"] = d["table"].cpu().numpy()
    bad = [(3, 0, 1, float("inf")), (90, 0, dim - 1, -float("inf")), (90, 1, 7, float("nan")), (199, 1, 7, 1.0),
           (150, 0, 1, float("inf")), (170, 0, 1, -float("inf"))]
    odd, zero = d["vc"].clone(), d["vc"].clone()
    want = torch.zeros((200, 4, dim), device="cuda")
    for at, head, e, value in bad:
        pos = ctx + at
        page, cell = int(d["table"][0, pos // 16]), pos % 16
        odd[page, head, e, cell] = value
        zero[page, head, e, cell] = value if value == 1.0 else 0.0
        if value != 1.0:
            want[at:, 2 * head:2 * head + 2, e] += value
    got, clean = _run(dict(d, vc=odd)), _run(dict(d, vc=zero))
    finite = want == 0
    assert torch.equal(got[finite], clean[finite])
    assert torch.equal(torch.nan_to_num(got[~finite].float(), 12345.0), torch.nan_to_num(want[~finite], 12345.0))


@pytest.mark.parametrize("dim", [64, 72, 128, 192, 256])
def test_every_number_of_tiles(dim):
    """Lengths around each multiple of the keys that are multiplied at a time, up to where the loop's
    first, middle and last rounds have all run."""
    lens = [1, 31, 32, 33, 63, 64, 65, 96, 97, 127, 129, 191, 193, 255, 257, 321, 384, 449, 513, 577]
    d = _long([n - 1 for n in lens], [1] * len(lens), 4, 2, dim, 8, "bfloat16", seed=dim)
    _check_long(d, _run(dict(d, table=d["table"].cpu().numpy())))


@pytest.mark.parametrize("shape", [
    # tiles of about 10, 16, 18, 21, 27 and 126 parts, and a long request beside short ones
    ([3000], [100], 32, 8, 128, 16, "bfloat16"),
    ([4000], [64], 32, 8, 128, 16, "float16"),
    ([20000], [64], 48, 12, 128, 16, "bfloat16"),
    ([9000], [30], 12, 12, 128, 32, "bfloat16"),
    ([20000], [64], 36, 9, 64, 16, "float16"),
    ([16000], [26], 3, 1, 128, 64, "bfloat16"),
    ([16000, 900, 40], [26, 30, 3], 3, 1, 80, 16, "bfloat16"),
    ([16000], [20], 8, 2, 256, 16, "bfloat16"),
])
def test_joins_of_few_and_many_parts(shape):
    """One thread for all parts of a row, or a quarter each; the same on every run."""
    import torch
    d = _long(*shape, seed=70)
    run = lambda: dgt.dgt_chunk_attention(d["q"], d["kc"], d["vc"], d["table"], _i32(d["ctx"]), _i32(d["cu"]))
    out = run()
    _check_long(d, out)
    assert torch.equal(run().view(torch.int16), out.view(torch.int16))
