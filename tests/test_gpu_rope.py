"""Norms, rotation and store against the 64-bit oracle.

Tolerance: one rounding to the 16-bit type, u |y| (2^-8, fp16 2^-11) and half a subnormal step, plus what
fp32 adds before it.  With n the head's norm factor (1 without norms) and m = |x^| of the pair together:
the sum of squares of dim terms and the square root are off by (dim + 4) 2^-24 relative, of which a result
takes half; two products, the weight and the sum 4 * 2^-24; cosines 2^-22 (their argument's rounding and the
series), so (dim / 2 + 10) 2^-24 m is enough."""

import numpy as np
import pytest

import decode_gemm_tile_amd as dgt
from oracle import serving

pytestmark = pytest.mark.gpu


def _i32(a):
    import torch
    return torch.from_numpy(np.ascontiguousarray(np.asarray(a, np.int32))).to("cuda")


def _make(seed, tokens, heads, kv, dim, block, source, cache, pairs, norms=(True, True), far=5000):
    import torch
    g = torch.Generator().manual_seed(seed)
    rng = np.random.default_rng(seed)
    cache = getattr(torch, cache)
    source = cache if source == "same" else torch.float32
    blocks = tokens // block + 5
    slots = rng.permutation(blocks * block)[:tokens]
    if seed % 2:  # whole runs of slots as prompts have them
        slots = (np.arange(tokens) + 3 * block // 2) % (blocks * block)
    positions = rng.integers(0, far, tokens)
    qkv = (torch.randn((tokens, (heads + 2 * kv), dim), generator=g) * 2).to(source)
    w = [torch.rand(dim, generator=g) + 0.5 if on else None for on in norms]
    freqs = 10000.0 ** -(np.arange(pairs) / max(pairs, 1))
    kc = torch.randn((blocks, kv, block, dim), generator=g).to(cache)
    vc = torch.randn((blocks, kv, dim, block), generator=g).to(cache)
    return dict(qkv=qkv, heads=heads, kv=kv, positions=positions, slots=slots, w=w, freqs=freqs, kc=kc, vc=vc,
                block=block)


def _run(d, **kw):
    import torch
    dev = lambda t: None if t is None else t.cuda()
    h, kv, x = d["heads"], d["kv"], d["qkv"].cuda()
    kc, vc = d["kc"].cuda(), d["vc"].cuda()
    freqs = torch.from_numpy(np.asarray(d["freqs"], np.float64)).cuda()
    q = dgt.dgt_rope_store(x[:, :h], x[:, h:h + kv], x[:, h + kv:], _i32(d["positions"]), _i32(d["slots"]), freqs, kc,
                           vc, q_weight=dev(d["w"][0]), k_weight=dev(d["w"][1]), **kw)
    torch.cuda.synchronize()
    return q, kc, vc


def _close(got, x, d, weight, rows, interleaved):
    ref = serving.rope(x[rows], d["positions"][rows], d["freqs"], weight, 1e-6, interleaved)
    dim, pairs = x.shape[2], len(d["freqs"])
    hat = serving.rope(x[rows], d["positions"][rows], [], weight, 1e-6)
    size = np.abs(hat)
    if interleaved:
        for i in range(pairs):
            size[:, :, 2 * i] = size[:, :, 2 * i + 1] = size[:, :, 2 * i] + size[:, :, 2 * i + 1]
    else:
        both = size[:, :, :pairs] + size[:, :, pairs:2 * pairs]
        size[:, :, :pairs], size[:, :, pairs:2 * pairs] = both, both
    u, low = (2.0 ** -8, 0.0) if "bfloat16" in str(d["kc"].dtype) else (2.0 ** -11, 2.0 ** -25)
    tol = u * np.abs(ref) + low + (dim / 2 + 10) * 2.0 ** -24 * size * (1 + u)
    err = np.abs(got - ref)
    assert (err <= tol).all(), float((err - tol).max())


def _check(d, q, kc, vc, interleaved=False):
    h, kv, block, blocks = d["heads"], d["kv"], d["block"], d["kc"].shape[0]
    x = d["qkv"].double().numpy()
    f = lambda t: None if t is None else t.double().numpy()
    live = np.nonzero(np.asarray(d["positions"]) >= 0)[0]
    _close(q.double().cpu().numpy()[live], x[:, :h], d, f(d["w"][0]), live, interleaved)
    slots = np.asarray(d["slots"])
    rows = np.array([t for t in live if 0 <= slots[t] < blocks * block], int)
    page, cell = slots[rows] // block, slots[rows] % block
    _close(kc.double().cpu().numpy()[page, :, cell], x[:, h:h + kv], d, f(d["w"][1]), rows, interleaved)
    # values: rounded to nearest even; and every other cell as it was
    vc0, kc0 = d["vc"].clone(), d["kc"].clone()
    vc0[page, :, :, cell] = d["qkv"][rows][:, h + kv:].to(vc0.dtype)
    kc0[page, :, cell] = kc.cpu()[page, :, cell]
    import torch
    assert torch.equal(vc.cpu().view(torch.int16), vc0.view(torch.int16))
    assert torch.equal(kc.cpu().view(torch.int16), kc0.view(torch.int16))


SHAPES = [  # tokens, heads, kv, dim, block, pairs
    (1, 1, 1, 64, 16, 32),
    (1, 32, 8, 128, 16, 64),
    (5, 8, 2, 128, 16, 64),
    (9, 3, 3, 80, 8, 40),
    (67, 4, 2, 128, 32, 32),
    (64, 2, 1, 64, 64, 16),
    (130, 6, 2, 72, 16, 36),
    (33, 5, 1, 256, 16, 128),
    (40, 2, 2, 200, 16, 100),
    (21, 4, 4, 8, 8, 4),
    (17, 2, 1, 24, 16, 5),
    (12, 2, 1, 128, 1024, 0),
    (300, 7, 1, 136, 16, 3),
]


@pytest.mark.parametrize("cache", ["bfloat16", "float16"])
@pytest.mark.parametrize("source", ["f32", "same"])
@pytest.mark.parametrize("interleaved", [False, True], ids=["halves", "pairs"])
@pytest.mark.parametrize("i", range(len(SHAPES)))
def test_rope_against_oracle(i, interleaved, source, cache):
    tokens, heads, kv, dim, block, pairs = SHAPES[i]
    d = _make(i + interleaved, tokens, heads, kv, dim, block, source, cache, pairs,
              norms=[(True, True), (False, False), (True, False), (False, True)][i % 4])
    _check(d, *_run(d, interleaved=interleaved), interleaved=interleaved)


def test_far_positions():
    """Angles of positions up to 2^31 - 1 are formed in 64 bits: 2^31 turns by 2^-53 of a turn each."""
    d = _make(3, 40, 2, 1, 128, 16, "f32", "float16", 64, far=2 ** 31 - 1)
    _check(d, *_run(d))


def test_many_tokens():
    import torch
    d = _make(5, 1500, 3, 1, 64, 16, "f32", "bfloat16", 32)
    _check(d, *_run(d))


def test_skipped_rows():
    """A negative position skips a row, also its query; a slot outside the pool only its key and value."""
    import torch
    d = _make(2, 70, 4, 2, 128, 16, "f32", "bfloat16", 64)
    d["positions"][::7] = -1
    d["slots"][3::5] = -1
    d["slots"][4::10] = d["kc"].shape[0] * 16
    d["slots"][9::20] = 2 ** 31 - 1
    out = torch.full((70, 4, 128), 9.0, dtype=torch.bfloat16, device="cuda")
    q, kc, vc = _run(d, q_out=out)
    assert q is out and bool((out[::7] == 9.0).all())
    _check(d, q, kc, vc)


def test_strides_alignment_and_streams():
    """Rows and heads of any stride, starts that are not 16-byte aligned, another stream."""
    import torch
    for off in (0, 1):
        d = _make(4 + off, 45, 4, 2, 80, 16, "f32", "bfloat16", 40)
        x = d["qkv"].cuda()
        flat = torch.full((45 * 1000 + off,), float("nan"), device="cuda")
        wide = flat[off:].view(45, 1000)
        q = wide[:, :4 * 88].view(45, 4, 88)[:, :, :80]
        k = wide[:, 400:600].view(45, 2, 100)[:, :, 3:83]
        v = wide[:, 700:].view(45, 2, 150)[:, :, 7:87]
        q.copy_(x[:, :4]), k.copy_(x[:, 4:6]), v.copy_(x[:, 6:])
        out = torch.full((45, 9, 96), 2.0, dtype=torch.bfloat16, device="cuda")[:, 1:5, 8:88]
        kc, vc, w = d["kc"].cuda(), d["vc"].cuda(), [t.cuda() for t in d["w"]]
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        dgt.dgt_rope_store(q, k, v, _i32(d["positions"]), _i32(d["slots"]), torch.from_numpy(d["freqs"]).cuda(), kc, vc,
                           q_weight=w[0], k_weight=w[1], q_out=out, stream=side)
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize()
        _check(d, out, kc, vc)


def test_a_bad_head_stays_alone():
    """NaN and infinity in one head's row leave the other heads and rows as they were."""
    import torch
    d = _make(6, 20, 4, 2, 64, 16, "f32", "bfloat16", 32)
    q0, kc0, _ = _run(d)
    d["qkv"][3, 1, 5], d["qkv"][4, 4, 6] = float("nan"), float("inf")
    q, kc, _ = _run(d)
    keep = torch.ones((20, 4), dtype=torch.bool)
    keep[3, 1] = False
    assert torch.equal(q.cpu()[keep], q0.cpu()[keep]) and bool(q[3, 1].isnan().all())
    page, cell = d["slots"][4] // 16, d["slots"][4] % 16
    kc0[page, 0, cell] = kc[page, 0, cell]
    assert torch.equal(kc.view(torch.int16), kc0.view(torch.int16))


def test_captured_and_replayed():
    import torch
    d = _make(8, 30, 4, 2, 128, 16, "f32", "bfloat16", 64)
    x, kc, vc, w = d["qkv"].cuda(), d["kc"].cuda(), d["vc"].cuda(), [t.cuda() for t in d["w"]]
    pos, slots, freqs = _i32(d["positions"]), _i32(d["slots"]), torch.from_numpy(d["freqs"]).cuda()
    q = torch.zeros((30, 4, 128), dtype=torch.bfloat16, device="cuda")
    run = lambda: dgt.dgt_rope_store(x[:, :4], x[:, 4:6], x[:, 6:], pos, slots, freqs, kc, vc, q_weight=w[0],
                                     k_weight=w[1], q_out=q)
    run()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for step in range(3):
        d["positions"] = d["positions"] + 100 * step
        pos.copy_(_i32(d["positions"]))
        q.zero_(), kc.copy_(d["kc"]), vc.copy_(d["vc"])
        graph.replay()
        torch.cuda.synchronize()
        _check(d, q, kc, vc)


def test_no_tokens():
    import torch
    d = _make(1, 3, 2, 1, 64, 16, "f32", "bfloat16", 32)
    d.update(qkv=d["qkv"][:0], positions=[], slots=[])
    q, kc, _ = _run(d)
    assert q.shape == (0, 2, 64) and torch.equal(kc.cpu(), d["kc"])
