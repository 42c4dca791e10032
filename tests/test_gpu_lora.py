"""Low-rank adapters against the 64-bit oracle.

Tolerance: the products of bf16 values are exact in fp32, so the error of
out = y + s (x A^T) B^T is that of its fp32 sums.  With S the same sum over
absolute values, adding K + rank terms in any order and scaling is off by at most
(K + rank + 40) * 2^-24 * S (40 covers the pieces of K and the waves), and adding
y rounds once: 2^-24 * |out| more."""

import numpy as np
import pytest

import decode_gemm_tile_amd as dgt
from oracle import serving

pytestmark = pytest.mark.gpu


def _make(seed, new, n, k, rank, adapters, ids=None, integers=False):
    import torch
    g = torch.Generator().manual_seed(seed)
    rng = np.random.default_rng(seed)
    tokens = int(sum(new))
    if integers:  # every sum below 2^24: exact in fp32 whatever the order
        def draw(shape, hi):
            return torch.randint(-hi, hi + 1, shape, generator=g).float()
        x, a, b = draw((tokens, k), 2), draw((adapters, rank, k), 1), draw((adapters, n, rank), 1)
        y, scaling = draw((tokens, n), 100), torch.randint(0, 3, (adapters,), generator=g) + 0.5
    else:
        x, a = torch.randn((tokens, k), generator=g), torch.randn((adapters, rank, k), generator=g) * k ** -0.5
        b, y = torch.randn((adapters, n, rank), generator=g), torch.randn((tokens, n), generator=g)
        scaling = torch.rand(adapters, generator=g) + 0.5
    ids = rng.integers(-1, adapters, len(new)) if ids is None else np.asarray(ids)
    cu = np.concatenate([[0], np.cumsum(new)])
    bf = lambda t: t.to(torch.bfloat16)
    return dict(y=y, x=bf(x), a=bf(a), b=bf(b), scaling=scaling.float(), ids=ids, cu=cu)


def _dev(d):
    import torch
    i32 = lambda v: torch.from_numpy(np.asarray(v, np.int32)).cuda()
    return (d["y"].cuda(), d["x"].cuda(), d["a"].cuda(), d["b"].cuda(), d["scaling"].cuda(), i32(d["ids"]),
            i32(d["cu"]))


def _oracle(d):
    f = lambda t: t.double().numpy()
    return serving.lora_add(f(d["y"]), f(d["x"]), f(d["a"]), f(d["b"]), f(d["scaling"]), d["ids"], d["cu"])


def _check(d, got):
    ref, size = _oracle(d)
    k, rank = d["x"].shape[1], d["a"].shape[1]
    tol = (k + rank + 40) * 2.0 ** -24 * size + 2.0 ** -24 * np.abs(ref)
    err = np.abs(got.double().cpu().numpy() - ref)
    assert (err <= tol).all(), float((err - tol).max())


SHAPES = [  # new tokens of each request, n, k, rank, adapters
    ([1], 128, 64, 8, 1),
    ([1], 1, 8, 8, 1),
    ([1] * 7, 257, 520, 16, 3),
    ([3, 0, 1, 17, 2], 100, 1000, 24, 2),
    ([16, 33, 5], 640, 256, 40, 4),
    ([70, 1, 129], 300, 4104, 64, 2),
    ([8, 9], 513, 96, 72, 2),
    ([200, 40], 130, 2048, 136, 2),
    ([5, 64, 1], 65, 512, 256, 3),
    ([2] * 130, 96, 128, 16, 20),
]


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "-".join(str(v) if not isinstance(v, list) else str(sum(v)) for v in s))
def test_lora_against_oracle(shape):
    import torch
    new, n, k, rank, adapters = shape
    d = _make(sum(new) + n, new, n, k, rank, adapters, ids=[i % adapters for i in range(len(new))])
    y, *rest = _dev(d)
    out = torch.full_like(y, float("nan"))
    got = dgt.dgt_lora_add(y, *rest, out=out)
    assert got is out
    _check(d, got)
    assert torch.equal(y.cpu(), d["y"])


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: str(s[1:]))
def test_lora_of_integers_is_exact(shape):
    new, n, k, rank, adapters = shape
    # |x A^T| <= 2k and |... B^T| <= 2k * rank * 2.5 + 100 < 2^23 for these shapes, in halves below 2^24
    assert 2 * k * rank * 2.5 + 100 < 2 ** 23
    d = _make(7, new, n, k, rank, adapters, integers=True)
    y, *rest = _dev(d)
    got = dgt.dgt_lora_add(y, *rest)
    assert got is y
    assert np.array_equal(got.double().cpu().numpy(), _oracle(d)[0])


def test_lora_ids_without_adapter():
    """Ids of -1, of the count and far outside: rows stay y, in place and beside it."""
    import torch
    d = _make(3, [2, 20, 3, 1, 9], 200, 256, 16, 2, ids=[0, -1, 2, 2 ** 31 - 1, 1])
    y, *rest = _dev(d)
    out = dgt.dgt_lora_add(y, *rest, out=torch.full_like(y, float("nan")))
    d["ids"] = np.array([0, -1, -1, -1, 1])
    _check(d, out)
    assert torch.equal(out[2:26].cpu(), d["y"][2:26])
    dgt.dgt_lora_add(y, *rest)
    assert torch.equal(y, out)


def test_lora_rows_of_no_request():
    """Rows past cu[-1] come back as y; no request and no adapter at all too."""
    import torch
    d = _make(4, [5, 3], 96, 128, 8, 2, ids=[1, 0])
    pad = torch.randn((30, 96))
    y, x, *rest = _dev(d)
    y = torch.cat([y, pad.cuda()])
    x = torch.cat([x, torch.full((30, 128), float("nan"), dtype=torch.bfloat16, device="cuda")])
    out = dgt.dgt_lora_add(y, x, *rest, out=torch.full_like(y, float("nan")))
    _check(d, out[:8])
    assert torch.equal(out[8:].cpu(), pad)
    a, b, s, ids, cu = rest
    none = torch.zeros(0, dtype=torch.int32, device="cuda")
    out = dgt.dgt_lora_add(y, x, a, b, s, none, cu[:1], out=torch.full_like(y, float("nan")))
    assert torch.equal(out, y)
    out = dgt.dgt_lora_add(y, x, a[:0], b[:0], s[:0], ids, cu, out=torch.full_like(y, float("nan")))
    assert torch.equal(out, y)
    assert dgt.dgt_lora_add(y[:0], x[:0], *rest[:4], torch.zeros(3, dtype=torch.int32, device="cuda")).numel() == 0


def test_lora_strided_rows():
    """x, y and out as column ranges of wider tensors; the columns beside them stay."""
    import torch
    d = _make(5, [1, 40, 3], 120, 264, 16, 3)
    _, _, *rest = _dev(d)
    wide_x = torch.full((44, 264 + 16), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide_y = torch.full((44, 300), 7.0, device="cuda")
    wide_o = torch.full((44, 131), 9.0, device="cuda")
    wide_x[:, 8:272], wide_y[:, 100:220] = d["x"].cuda(), d["y"].cuda()
    out = dgt.dgt_lora_add(wide_y[:, 100:220], wide_x[:, 8:272], *rest, out=wide_o[:, 5:125])
    _check(d, out)
    assert (wide_o[:, :5] == 9).all() and (wide_o[:, 125:] == 9).all()
    dgt.dgt_lora_add(wide_y[:, 100:220], wide_x[:, 8:272], *rest)
    assert torch.equal(wide_y[:, 100:220], out)
    assert (wide_y[:, :100] == 7).all() and (wide_y[:, 220:] == 7).all()


def test_lora_single_row_of_any_stride():
    """The stride of a dimension of size one means nothing: a transposed column is a row."""
    import torch
    d = _make(14, [1], 130, 64, 16, 2, ids=[1])
    y, x, *rest = _dev(d)
    want = dgt.dgt_lora_add(y, x, *rest, out=torch.empty_like(y))
    _check(d, want)
    column = lambda t: t.clone().as_strided(t.shape, (1, 1))  # as (n, 1) transposed has it
    for y1, x1, out in ((column(y), x, None), (y, x.as_strided((1, 64), (3, 1)), column(y)),
                        (column(y), column(x), torch.empty_like(y))):
        assert y1.is_contiguous() and x1.is_contiguous()
        assert torch.equal(dgt.dgt_lora_add(y1, x1, *rest, out=out), want)


def test_lora_nan_stays_in_its_rows():
    """A NaN or infinity in one request's x or adapter does not reach the others."""
    import torch
    d = _make(6, [1, 1, 18, 1], 150, 128, 16, 3, ids=[0, 1, 2, 0])
    d["x"][1, 5] = float("inf")
    d["a"][2, 3, 7] = float("nan")
    y, *rest = _dev(d)
    out = dgt.dgt_lora_add(y, *rest, out=torch.empty_like(y)).cpu()
    assert not torch.isfinite(out[1]).any() and torch.isnan(out[2:20]).all()
    keep = [0, 20]
    ref, _ = _oracle(d)
    assert np.allclose(out[keep].numpy(), ref[keep], atol=1e-4)


def _check_non_finite(d, got):
    """Infinities and NaN where the definition has them, all else within the tolerance."""
    with np.errstate(invalid="ignore"):
        ref, size = _oracle(d)
    got = got.double().cpu().numpy()
    assert np.array_equal(np.isnan(got), np.isnan(ref))
    assert np.array_equal(np.isposinf(got), np.isposinf(ref)) and np.array_equal(np.isneginf(got), np.isneginf(ref))
    k, rank = d["x"].shape[1], d["a"].shape[1]
    ok = np.isfinite(ref)
    tol = (k + rank + 40) * 2.0 ** -24 * size[ok] + 2.0 ** -24 * np.abs(ref[ok])
    assert (np.abs(got[ok] - ref[ok]) <= tol).all()


@pytest.mark.parametrize("integers", [False, True], ids=["reals", "integers"])
@pytest.mark.parametrize("new,rank", [([1, 5, 3], 16), ([40, 33], 72)])
def test_lora_infinite_weights(new, rank, integers):
    """An infinity of B makes its column infinite with the sign of the shrunk value, whichever
    bits that has (integers leave the lower parts zero); two of different signs, or one times
    zero, make NaN; the other columns are as ever."""
    d = _make(12, new, 150, 256, rank, 2, ids=[0, 1, 0][:len(new)], integers=integers)
    inf = float("inf")
    d["b"][0, 3, 2], d["b"][0, 77, 5], d["b"][1, 149, rank - 1], d["b"][1, 0, 0] = inf, -inf, inf, inf
    d["b"][0, 100, 1], d["b"][0, 100, 9] = inf, -inf
    d["b"][1, 50, 4] = float("nan")
    y, *rest = _dev(d)
    out = dgt.dgt_lora_add(y, *rest)
    _check_non_finite(d, out)
    assert out.isinf().any() and out.isnan().any()


def test_lora_values_beside_the_largest():
    """A shrunk value that no bf16 value is near from above: its products with small weights
    are finite, with zeros zero."""
    import torch
    d = _make(13, [1, 2], 40, 64, 8, 1, ids=[0, 0])
    d["x"].zero_(), d["a"].zero_()
    d["x"][:, :2] = torch.tensor([[1.0, 1.0], [1.0, 0.0], [-1.0, -1.0]])
    d["a"][0, 4, :2] = torch.tensor([3.375, 0.0234375])
    d["scaling"][:] = 1e38
    d["b"] = (d["b"].float() * 2.0 ** -100).to(torch.bfloat16)
    d["b"][0, ::3] = 0
    # (1e38 is not exact in fp32: the oracle takes the value that the operator gets)
    y, *rest = _dev(d)
    out = dgt.dgt_lora_add(y, *rest)
    assert torch.isfinite(out).all()
    _check_non_finite(d, out)


def test_lora_garbage_offsets_stay_inside():
    """Offsets out of order or past the rows touch nothing outside; a sound call after it is right."""
    import torch
    d = _make(8, [4, 4, 4], 64, 64, 8, 2, ids=[0, 1, 0])
    y, x, a, b, s, ids, cu = _dev(d)
    ws = dgt.alloc_workspace(dgt.dgt_lora_workspace(12, 3, 64, 64, 8))
    for bad in ([0, 2 ** 31 - 1, 5, 12], [-7, 4, 2, -1], [9, 3, 1, 0], [12, 12, 12, 12]):
        guard = torch.full((14, 64), 3.0, device="cuda")
        dgt.dgt_lora_add(y, x, a, b, s, ids, torch.tensor(bad, dtype=torch.int32, device="cuda"),
                         out=guard[1:13], ws=ws)
        torch.cuda.synchronize()
        assert (guard[0] == 3).all() and (guard[13] == 3).all()
    _check(d, dgt.dgt_lora_add(y, x, a, b, s, ids, cu, out=torch.empty_like(y), ws=ws))


def test_lora_repeats_bit_for_bit_and_on_other_streams():
    import torch
    d = _make(9, [1] * 20 + [90], 1000, 4096, 32, 5)
    args = _dev(d)
    first = dgt.dgt_lora_add(*args, out=torch.empty_like(args[0]))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out = torch.empty_like(first)
    dgt.dgt_lora_add(*args, out=out, stream=s)
    s.synchronize()
    assert torch.equal(out, first)
    _check(d, first)


def test_lora_in_a_graph():
    import torch
    d = _make(10, [1, 2, 30], 384, 512, 16, 2, ids=[0, 1, 1])
    y, *rest = _dev(d)
    out, ws = torch.empty_like(y), dgt.alloc_workspace(dgt.dgt_lora_workspace(33, 3, 384, 512, 16))
    want = dgt.dgt_lora_add(y, *rest, out=out, ws=ws).clone()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dgt.dgt_lora_add(y, *rest, out=out, ws=ws)
    for scale in (1.0, 2.0, 0.5):
        out.fill_(float("nan"))
        y.copy_(d["y"].cuda() * scale)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.allclose(out - y, want - d["y"].cuda(), atol=1e-5)
