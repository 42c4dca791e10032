"""Verification of drafts against the 64-bit oracle: paths, counts and next tokens are equal.

Inputs are drawn once; a draw in which a uniform number lies within 1e-9 of a border would not say
anything, and the oracle's own checks (tests/test_oracle_step.py) hold the definition."""

import numpy as np
import pytest

import decode_gemm_tile_amd as dgt
from oracle import serving

pytestmark = pytest.mark.gpu


def _i32(a):
    import torch
    return torch.from_numpy(np.ascontiguousarray(np.asarray(a, np.int32))).to("cuda")


def _f32(a):
    import torch
    return torch.from_numpy(np.ascontiguousarray(np.asarray(a, np.float32))).to("cuda")


def _make(seed, new, vocab, tree=False, probs=False, dtype="float32", temperature=None, boost=4.0):
    import torch
    rng = np.random.default_rng(seed)
    tokens = int(sum(new))
    logits = rng.normal(size=(tokens, vocab)) * 2
    parents = np.concatenate([[-1] * min(n, 1) + [int(rng.integers(max(-1 if tree > 1 else 0, i - 6), i)) for i in range(1, n)]
                              for n in new] + [[]]).astype(int) if tree else None
    cu = np.concatenate([[0], np.cumsum(new)]).astype(int)
    draft = rng.integers(0, vocab, tokens)
    q = None
    if probs:
        z = logits * 1.1 + rng.normal(size=logits.shape) * 0.7
        q = np.exp(z - z.max(1, keepdims=True))
        q = (q / q.sum(1, keepdims=True)).astype(np.float32)
    for b in range(len(new)):
        for i in range(1, new[b]):
            up = int(parents[cu[b] + i]) if tree else i - 1
            if up < 0:
                continue
            if probs:
                draft[cu[b] + i] = rng.choice(vocab, p=q[cu[b] + up].astype(float) / q[cu[b] + up].astype(float).sum())
            elif rng.random() < 0.8:
                logits[cu[b] + up, draft[cu[b] + i]] += boost + np.log(vocab) / 2
    logits = torch.from_numpy(logits).to(getattr(torch, dtype))
    heat = None if temperature is None else np.asarray(temperature, np.float32)
    return dict(logits=logits, draft=draft, cu=cu, new=list(new), parents=parents, probs=q, heat=heat,
                accept=rng.random(tokens).astype(np.float32), sample=rng.random(len(new)).astype(np.float32))


def _args(d):
    return ((d["logits"].cuda(), _i32(d["draft"]), _i32(d["cu"]), _f32(d["accept"]), _f32(d["sample"])),
            dict(parents=None if d["parents"] is None else _i32(d["parents"]),
                 draft_probs=None if d["probs"] is None else _f32(d["probs"]),
                 temperature=None if d["heat"] is None else _f32(d["heat"])))


def _run(d, **kw):
    import torch
    args, named = _args(d)
    v = dgt.dgt_verify(*args, **(named | kw))
    torch.cuda.synchronize()
    return v


def _oracle(d, b):
    s, e = int(d["cu"][b]), int(d["cu"][b + 1])
    part = lambda x: None if d[x] is None else d[x][s:e]
    return serving.verify(d["logits"][s:e].double().numpy(), d["draft"][s:e], d["accept"][s:e], d["sample"][b],
                          part("parents"), part("probs"), 1.0 if d["heat"] is None else d["heat"][b])


def _check(d, v):
    path, accepted, token = (x.cpu().numpy() for x in (v.path, v.accepted, v.next))
    lengths = []
    for b, n in enumerate(d["new"]):
        way, following = _oracle(d, b)
        s = int(d["cu"][b])
        assert path[s:s + n].tolist() == way + [-1] * (n - len(way)), b
        assert accepted[b] == len(way) and token[b] == following, (b, token[b], following)
        lengths.append(len(way))
    return lengths


CASES = [  # new, vocab
    ([1], 1), ([1], 17), ([4], 100), ([3, 0, 1, 7], 1000), ([9, 2], 4095), ([5], 4096), ([6, 6], 4097),
    ([2, 30, 5], 8192), ([12] * 5, 50001), ([70, 3], 2000), ([3], 130000), ([8] * 40, 700),
]


@pytest.mark.parametrize("dtype", ["float32", "bfloat16", "float16"])
@pytest.mark.parametrize("kind", ["chain", "probs", "tree", "forest"])
@pytest.mark.parametrize("i", range(len(CASES)))
def test_verify_against_oracle(i, kind, dtype):
    new, vocab = CASES[i]
    d = _make(10 * i, new, vocab, tree={"tree": 1, "forest": 2}.get(kind, 0), probs=kind == "probs", dtype=dtype)
    _check(d, _run(d))


@pytest.mark.parametrize("kind", ["chain", "probs", "tree"])
def test_temperatures(kind):
    """0 and below (and NaN): the most likely token; others divide the logits."""
    d = _make(5, [6] * 12, 900, tree=int(kind == "tree"), probs=kind == "probs",
              temperature=[0.0, -1.0, 0.3, 0.7, 1.0, 1.5, 4.0, 1e-3, 1e-30, 1e6, float("nan"), 0.05])
    _check(d, _run(d))


def test_paths_of_all_lengths():
    """Over many requests some paths end at once and some go to the end."""
    d = _make(6, [5] * 200, 300, probs=True)
    lengths = _check(d, _run(d))
    assert set(lengths) == {1, 2, 3, 4, 5}
    d = _make(7, [15] * 200, 300, tree=True)
    assert len(set(_check(d, _run(d)))) >= 5


def test_first_of_equal_logits():
    d = _make(8, [3, 2], 9000, temperature=[0, 0])
    d["logits"] = d["logits"].float().round().clamp(-3, 3)
    d["draft"][1] = int(d["logits"][0].argmax())
    _check(d, _run(d))


def test_excluded_tokens():
    """-inf excludes a token: it is never accepted and never follows; a row of -inf alone, with a NaN or
    with +inf ends the path and gives -1."""
    d = _make(9, [4] * 8, 5000)
    d["logits"][:, ::3] = float("-inf")
    d["logits"][:, 4096:] = float("-inf")  # a whole segment
    d["draft"][1::4] = 0
    v = _run(d)
    _check(d, v)
    following = v.next.cpu().numpy()
    assert (following % 3 != 0).all() and (following < 4096).all()
    d["logits"][0] = float("-inf")
    d["logits"][4, 17] = float("nan")
    d["logits"][8, 4500] = float("inf")
    for heat in (None, [0.0] * 8):
        d["heat"] = heat
        v = _run(d)
        _check(d, v)
        assert v.next[:3].tolist() == [-1] * 3 and v.accepted[:3].tolist() == [1] * 3


def test_refused_once_is_refused_again():
    """Siblings with one token, and drafts outside the vocabulary."""
    d = _make(11, [9] * 30, 60, tree=True)
    d["parents"] = np.tile([-1] + [0] * 8, 30)
    d["draft"] = np.random.default_rng(0).integers(0, 4, 270)
    d["draft"][5::9] = 60
    d["draft"][6::9] = -1
    lengths = _check(d, _run(d))
    assert 1 in lengths and 2 in lengths


def test_drafts_that_the_draft_model_excludes():
    """q(x) = 0 is accepted wherever p(x) > 0; q = p is always accepted; negative and NaN count as 0."""
    import torch
    d = _make(12, [3] * 20, 200, probs=True)
    d["probs"][::6] = 0.0
    d["probs"][1::6] = np.exp(serving.softmax(np.zeros(200)))
    d["probs"][2::9, 5] = float("nan")
    d["probs"][3::9, 7] = -0.5
    _check(d, _run(d))
    d = _make(13, [4] * 20, 200, probs=True)
    p = torch.softmax(d["logits"].double(), 1)
    d["probs"] = (p * 0.9999).float().numpy()
    assert set(_check(d, _run(d))) == {4}


@pytest.mark.parametrize("kind", ["chain", "tree", "probs"])
def test_borders_of_the_numbers(kind):
    """0 takes the first token that has a probability, and every draft that has one; the largest number below
    1 takes the last."""
    for accept, sample in ((0.0, 0.0), (0.0, 1 - 2.0 ** -24), (1 - 2.0 ** -24, 0.0), (1 - 2.0 ** -24, 1 - 2.0 ** -24)):
        d = _make(14, [4] * 6, 6000, tree=int(kind == "tree"), probs=kind == "probs")
        d["logits"][:, :100] = float("-inf")
        d["logits"][:, 5900:] = float("-inf")
        d["accept"][:], d["sample"][:] = accept, sample
        _check(d, _run(d))


def test_rows_behind_the_last_request_are_left():
    import torch
    d = _make(15, [3, 4], 500)
    d["logits"] = torch.cat([d["logits"], torch.full((5, 500), float("nan"))])
    d["draft"] = np.concatenate([d["draft"], [7] * 5])
    d["accept"] = np.concatenate([d["accept"], [0.5] * 5])
    out = dgt.Verified.empty(2, 12)
    out.path.fill_(77)
    v = _run(d, out=out)
    assert v is out and (out.path[7:] == 77).all()
    _check(d, v)


def test_strides_streams_and_workspace():
    import torch
    d = _make(16, [5, 1, 6], 4100, probs=True)
    wide = torch.full((12, 4203), float("nan"), device="cuda")
    wide[:, 3:4103] = d["logits"].cuda()
    q = torch.full((12, 4111), float("nan"), device="cuda")
    q[:, 1:4101] = _f32(d["probs"])
    args, named = _args(d)
    ws = torch.full((dgt.dgt_verify_workspace(12, 4100, 3),), 255, dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        v = dgt.dgt_verify(wide[:, 3:4103], *args[1:], **(named | dict(draft_probs=q[:, 1:4101])), ws=ws, stream=side)
        side.synchronize()
        _check(d, v)


def test_offsets_that_do_not_fit():
    """Offsets that fall or lie outside leave nothing written outside the arrays."""
    import torch
    d = _make(17, [6], 300, tree=True)
    args, named = _args(d)
    for cu in ([0, 2 ** 31 - 1], [-9, 4], [5, 1], [6, 6]):
        whole = torch.full((8,), 77, dtype=torch.int32, device="cuda")
        out = dgt.Verified.empty(1, 6)
        out.path = whole[1:7]
        dgt.dgt_verify(args[0], args[1], _i32(cu), *args[3:], **named, out=out)
        assert whole[0] == 77 and whole[7] == 77
    named["parents"] = _i32([5, 9, -7, 2 ** 31 - 1, 3, 0])  # links that are no tree's
    dgt.dgt_verify(*args, **named)
    torch.cuda.synchronize()


def test_captured_and_replayed():
    import torch
    for kind in ("tree", "probs"):
        d = _make(18, [7, 3, 9], 5000, tree=int(kind == "tree"), probs=kind == "probs")
        args, named = _args(d)
        ws = torch.zeros(dgt.dgt_verify_workspace(19, 5000, 3), dtype=torch.uint8, device="cuda")
        out = dgt.Verified.empty(3, 19)
        run = lambda: dgt.dgt_verify(*args, **named, out=out, ws=ws)
        run()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            run()
        rng = np.random.default_rng(1)
        for _ in range(4):
            d["accept"], d["sample"] = rng.random(19).astype(np.float32), rng.random(3).astype(np.float32)
            args[3].copy_(_f32(d["accept"])), args[4].copy_(_f32(d["sample"]))
            graph.replay()
            torch.cuda.synchronize()
            _check(d, out)


def test_distribution():
    """8000 requests of one chain and of one tree: what comes out first is distributed as the target's own
    samples, whatever the drafts.  A count of probability p stays within 6 sqrt(n p) of n p (and 6)."""
    import torch
    n, vocab = 8000, 12
    rng = np.random.default_rng(2)
    row = rng.normal(size=vocab) * 1.5
    p = serving.softmax(np.float32(row).astype(float))
    for kind in ("probs", "tree"):
        new = 2 if kind == "probs" else 4
        logits = torch.from_numpy(np.tile(np.float32(row), (n * new, 1)))
        q = serving.softmax(rng.normal(size=vocab))
        draft = rng.choice(vocab, size=n * new, p=q)
        if kind == "tree":  # distinct children
            draft = np.stack([rng.permutation(vocab)[:new] for _ in range(n)]).reshape(-1)
        d = dict(logits=logits, draft=draft, cu=np.arange(n + 1) * new, new=[new] * n, heat=None,
                 parents=np.tile([-1] + [0] * (new - 1), n) if kind == "tree" else None,
                 probs=np.tile(np.float32(q), (n * new, 1)) if kind == "probs" else None,
                 accept=rng.random(n * new).astype(np.float32), sample=rng.random(n).astype(np.float32))
        v = _run(d)
        path, accepted, token = (x.cpu().numpy() for x in (v.path, v.accepted, v.next))
        first = np.where(accepted > 1, draft.reshape(n, new)[np.arange(n), path.reshape(n, new)[:, 1].clip(0)], token)
        counts = np.bincount(first, minlength=vocab)
        assert (np.abs(counts - n * p) <= 6 * np.sqrt(n * p) + 6).all(), (kind, counts, n * p)


def test_no_rows():
    import torch
    d = _make(19, [], 50)
    v = _run(d)
    assert v.next.numel() == 0
    d = _make(19, [0, 0], 50, tree=True)
    v = _run(d)
    assert v.accepted.tolist() == [0, 0] and v.next.tolist() == [-1, -1]


@pytest.mark.parametrize("kind", ["chain", "probs", "tree"])
def test_an_infinite_temperature(kind):
    """All tokens weigh the same; the largest finite temperature comes close to it."""
    d = _make(8, [6] * 12, 900, tree=int(kind == "tree"), probs=kind == "probs",
              temperature=[float("inf"), 3.4e38] * 6)
    _check(d, _run(d))
    assert len(set(_run(d).next.tolist())) > 6  # not one most likely token after the other


def _beside(border, above):
    """float32 numbers next to their borders (in 64 bits), above or below, at least 2^-26 of the border and at
    most three of its last places away."""
    u = np.float32(border)
    for i, (b, up) in enumerate(zip(border, above)):
        while (float(u[i]) - b) * (1 if up else -1) < b * 2.0 ** -26:
            u[i] = np.nextafter(u[i], np.float32(2 if up else -1))
    far = np.abs(u.astype(float) - border) / border
    assert far.min() >= 2.0 ** -26 and far.max() <= 3 * 2.0 ** -23 and u.max() < 1
    return u


@pytest.mark.parametrize("dtype", ["float32", "bfloat16", "float16"])
@pytest.mark.parametrize("kind", ["chain", "probs", "tree"])
@pytest.mark.parametrize("vocab", [300, 5000, 50001, 130000])
def test_numbers_next_to_their_borders(vocab, kind, dtype):
    """A draft's number one last place from the border falls on the border's right side: sums over a vocabulary
    are 64-bit.  (Their weights are off by 2^-39, the numbers by 2^-26 at least.)"""
    n = 40 if vocab < 100000 else 16
    d = _make(30, [2] * n, vocab, probs=kind == "probs", dtype=dtype, temperature=np.linspace(0.5, 1.5, n))
    rng = np.random.default_rng(31)
    above = rng.random(n) < 0.5
    z = d["logits"].double().numpy()[::2] / d["heat"].astype(float)[:, None]
    p = np.exp(z - z.max(1, keepdims=True))
    p /= p.sum(1, keepdims=True)
    best = np.argsort(p, 1)[np.arange(n), -1 - rng.integers(1, 5, n)]
    d["draft"][1::2] = best
    border = p[np.arange(n), best]
    if kind == "probs":
        d["probs"][::2][np.arange(n), best] = q = np.float32(border * (1.1 + rng.random(n)))
        border = border / q.astype(float)
    if kind == "tree":
        d["parents"] = np.tile([-1, 0], n)
    d["accept"][1::2] = _beside(border, above)
    lengths = _check(d, _run(d))
    assert lengths == (2 - above).tolist()


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("levels", [1, 2, 4, 6])
def test_numbers_next_to_their_borders_behind_refused_siblings(levels, dtype):
    """What siblings leave of the mass, down to a millionth of it, keeps its bits: each takes about nine tenths of
    what is left, and the last one's number lies next to the border."""
    n, vocab = 30, 20000
    import torch
    rng = np.random.default_rng(33)
    new = levels + 2
    logits = rng.normal(size=(n * new, vocab)) * 2
    ids = np.stack([rng.permutation(vocab)[:levels + 1] for _ in range(n)])
    total = np.log(np.exp(logits[::new]).sum(1))
    for i in range(levels + 1):
        logits[np.arange(n) * new, ids[:, i]] = total + (levels - i) * np.log(10) + np.log(9)
    logits = torch.from_numpy(logits).to(getattr(torch, dtype))
    z = logits.double().numpy()[::new]
    p = np.exp(z - z.max(1, keepdims=True))
    border = np.zeros((n, levels + 1))
    for i in range(levels + 1):
        border[:, i] = p[np.arange(n), ids[:, i]] / p.sum(1)
        p[np.arange(n), ids[:, i]] = 0
    above = rng.random(n) < 0.5
    accept = np.full((n, new), 0.99, np.float32)
    assert border.max() < 0.98
    accept[:, -1] = _beside(border[:, -1], above)
    d = dict(logits=logits, draft=np.concatenate([np.zeros((n, 1), int), ids], 1).reshape(-1), new=[new] * n,
             cu=np.arange(n + 1) * new, parents=np.tile([-1] + [0] * (levels + 1), n), probs=None, heat=None,
             accept=accept.reshape(-1), sample=rng.random(n).astype(np.float32))
    lengths = _check(d, _run(d))
    assert lengths == (2 - above).tolist()


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("kind", ["chain", "tree", "probs"])
def test_masks_of_the_lowest_value(kind, dtype):
    """A mask of the type's lowest value excludes a token at an ordinary temperature; at an infinite one, which
    makes all tokens but those of -inf weigh the same, it does not; at a very large one it weighs what the
    formula says, also beside a logit as large, whose distance fp32 does not hold."""
    import torch
    low = float(torch.finfo(getattr(torch, dtype)).min)
    n, vocab = 24, 900
    for large, heats in ((False, [1.0, 1e-3]), (False, [float("inf")]), (False, [3.4e38, 1e38]),
                         (True, [float("inf"), 3.4e38, 1e38, 3e37])):
        d = _make(40, [3] * n, vocab, tree=int(kind == "tree"), probs=kind == "probs", dtype=dtype,
                  temperature=np.resize(heats, n))
        d["logits"][:, 5:600] = low
        d["logits"][:, 600:640] = float("-inf")
        if large:
            d["logits"][:, 640:700] = -low
        drafted = np.random.default_rng(41).integers(0, 700, 3 * n)
        d["draft"] = drafted
        if kind == "probs":
            d["probs"][:] = 1.0 / vocab
        _check(d, _run(d))


@pytest.mark.parametrize("kind", ["chain", "probs", "tree"])
@pytest.mark.parametrize("vocab", [700, 30000, 60000])
def test_paths_of_numbers_next_to_their_borders(vocab, kind):
    """Number after number next to its border, some requests greedy or with rows that end a path: paths go on
    behind a close one."""
    n, new = 24, 7
    heat = np.where(np.arange(n) % 8 == 7, 0.0, np.linspace(0.6, 1.4, n)).astype(np.float32)
    d = _make(50, [new] * n, vocab, probs=kind == "probs", temperature=heat)
    rng = np.random.default_rng(51)
    d["parents"] = np.tile([-1, 0, 0, 2, 2, 2, 5], n) if kind == "tree" else None
    up = np.tile([-1, 0, 0, 2, 2, 2, 5] if kind == "tree" else np.arange(-1, new - 1), (n, 1))
    # where the path is to go: of a tree to 2 (past 1), 5 (past 3 and 4), 6; of a chain down to a row of its own
    stop = rng.integers(1, new + 1, n)
    refused = np.tile([False, True, False, True, True, False, False], (n, 1)) if kind == "tree" else (
        np.arange(new) >= stop[:, None])
    refused[::5, -1] = True
    logits = d["logits"].numpy().reshape(n, new, vocab)
    logits[3, 2, 17] = np.nan
    draft, accept = d["draft"].reshape(n, new), d["accept"].reshape(n, new)
    for b in range(n):
        left = {}
        for i in range(1, new):
            row = logits[b, up[b, i]].astype(float)
            if not np.isfinite(row).all() or heat[b] <= 0:
                draft[b, i] = np.nanargmax(row) if not refused[b, i] else np.nanargmin(row)
                continue
            p = np.exp((row - row.max()) / float(heat[b]))
            p /= p.sum()
            gone = left.setdefault(up[b, i], [])
            draft[b, i] = x = np.argsort(p)[-1 - len(gone) - int(rng.integers(0, 2)) * 3]
            border = p[x] / np.delete(p, gone).sum()
            if kind == "probs":
                d["probs"][b * new + up[b, i], x] = q = np.float32(p[x] * 1.3)
                border = p[x] / float(q)
            accept[b, i] = _beside(np.array([border]), [refused[b, i]])[0]
            gone.append(x)
    lengths = _check(d, _run(d))
    live = [b for b in range(n) if b != 3]
    if kind == "tree":
        assert [lengths[b] for b in live] == [3 if refused[b, -1] else 4 for b in live]
    else:
        assert [lengths[b] for b in live] == [int(np.argmax(np.append(refused[b], True))) for b in live]


def test_rows_that_the_path_passes_by():
    """Many trees whose rows are read and passed by while the paths go on: every run gives the same, and what the
    definition says."""
    d = _make(60, [27] * 60 + [70] * 4, 12300, tree=True)
    args, named = _args(d)
    ws = dgt.alloc_workspace(dgt.dgt_verify_workspace(1900, 12300, 64))
    _check(d, _run(d, ws=ws))
    first = _run(d, ws=ws)
    for _ in range(20):
        v = dgt.dgt_verify(*args, **named, ws=ws)
        assert v.path.equal(first.path) and v.accepted.equal(first.accepted) and v.next.equal(first.next)
