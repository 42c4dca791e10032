"""Measured cases of the operators around a verify step: queries, keys and values from
the projection's rows into the attention's queries and the paged cache (norms and
rotation on the way), verification of drafted tokens against the target's logits,
moving, forking and freeing pages, and attention of a chunk of new tokens.

``run`` computes a case either with the library's kernels (``own = True``) or in a
plain form of elementary torch operations (``own = False``); both take the state that
``prepare`` makes.  ``exact`` computes the same outputs from the definitions in 64 bits.

Shapes.  A request b holds ctx[b] tokens in the cache and brings new[b] tokens to the
step; the new tokens of all requests lie one after another in T rows, request b in rows
cu[b] .. cu[b + 1] - 1.  Key pages are [layers, blocks, heads, block, dim]; value pages
are transposed, [layers, blocks, heads, dim, block].  Lengths form a ladder from short to
the stated maximum, dealt to the requests in an order drawn from the seed, so a case's
work is the same for every seed.
"""

import math
import random

import numpy as np
import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def listed():
    return [
        # One decoding user: the row of one token, half precision throughout, pairs side by
        # side, a part of each head turned; latency only.
        {"name": "rope_token", "op": "rope", "requests": 1, "ctx": 1900, "new": 1, "heads": 16, "kv_heads": 4,
         "dim": 64, "pairs": 16, "interleaved": True, "norms": False, "block": 32, "source": "same", "cache": "f16"},
        # Prompts of uneven lengths, out of the fp32 rows of the fused qkv projection, with
        # norms of queries and keys.
        {"name": "rope_prompts", "op": "rope", "requests": 7, "ctx": 60000, "new": 2047, "heads": 32, "kv_heads": 8,
         "dim": 128, "pairs": 64, "interleaved": False, "norms": True, "block": 16, "source": "f32", "cache": "bf16"},
        # A few users with short chains from a small draft model, a small vocabulary; latency.
        {"name": "verify_chains", "op": "verify", "requests": 5, "new": 5, "tree": False, "probs": True,
         "vocab": 32000, "logits": "f32", "greedy": False},
        # A decoding batch with chains from a draft model that returns its probabilities.
        {"name": "verify_batch", "op": "verify", "requests": 96, "new": 7, "tree": False, "probs": True,
         "vocab": 128000, "logits": "bf16", "greedy": False},
        # Trees of up to 27 nodes (children are the draft's best tokens) for a medium batch;
        # some requests are greedy.
        {"name": "verify_trees", "op": "verify", "requests": 64, "new": 27, "tree": True, "probs": False,
         "vocab": 128000, "logits": "f32", "greedy": True},
        # What a small batch keeps of its trees, one layer's cache.
        {"name": "keep_few", "op": "keep", "requests": 4, "ctx": 900, "new": 13, "layers": 1, "kv_heads": 8,
         "dim": 128, "block": 16, "cache": "bf16"},
        # A large batch with trees of up to 61 nodes, several layers in one call.
        {"name": "keep_trees", "op": "keep", "requests": 128, "ctx": 600, "new": 61, "layers": 4, "kv_heads": 8,
         "dim": 128, "block": 16, "cache": "bf16"},
        # One prompt answered three times: its pages are shared, the last one is copied; and
        # the answers dropped again.
        {"name": "branch_few", "op": "branch", "requests": 1, "children": 3, "ctx": 1003, "layers": 2,
         "kv_heads": 8, "dim": 128, "block": 16, "cache": "bf16"},
        # Beams of a batch: every request forked into four, long pages; and dropped again.
        {"name": "branch_beams", "op": "branch", "requests": 48, "children": 4, "ctx": 3001, "layers": 4,
         "kv_heads": 8, "dim": 128, "block": 64, "cache": "bf16"},
        # A short chunk of a long prompt, one user: the cache is split over the card.
        {"name": "chunk_one", "op": "chunk", "requests": 1, "ctx": 3000, "new": 100, "heads": 32, "kv_heads": 8,
         "dim": 128, "block": 16, "cache": "bf16"},
        # A batch of chunks of uneven lengths behind uneven contexts, half precision, three
        # query heads to a key head.
        {"name": "chunk_mixed", "op": "chunk", "requests": 24, "ctx": 6000, "new": 700, "heads": 24, "kv_heads": 8,
         "dim": 128, "block": 32, "cache": "f16"},
        # Whole prompts.
        {"name": "chunk_prompts", "op": "chunk", "requests": 3, "ctx": 500, "new": 8190, "heads": 32, "kv_heads": 8,
         "dim": 128, "block": 16, "cache": "bf16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "verify", "keep", "branch", "chunk", "chunk"])
    cache, block = rng.choice(["bf16", "bf16", "f16"]), rng.choice([16, 32, 64])
    if op == "rope":
        kv, requests, dim = rng.choice([1, 2, 3, 8]), _log(rng, 1, 64), rng.choice([64, 80, 128, 128])
        return {"op": op, "requests": requests, "ctx": _log(rng, 1, 60000),
                "new": max(1, min(2047, _log(rng, 1, 8000) // requests)), "heads": kv * rng.choice([1, 4]),
                "kv_heads": kv, "dim": dim, "pairs": rng.choice([dim // 2, dim // 2, dim // 4]),
                "interleaved": rng.random() < 0.4, "norms": rng.random() < 0.6, "block": block,
                "source": rng.choice(["f32", "f32", "same"]), "cache": cache}
    if op == "verify":
        tree = rng.random() < 0.5
        requests, vocab = _log(rng, 1, 96), rng.choice([_log(rng, 500, 128000), 32000, 128000])
        new = max(1, min(61 if tree else 9, _log(rng, 2, 1800) // requests))
        return {"op": op, "requests": requests, "new": new, "tree": tree,
                "probs": not tree and rng.random() < 0.7, "vocab": vocab,
                "logits": rng.choice(["f32", "f32", "bf16", "f16"]), "greedy": rng.random() < 0.3}
    kv, dim = rng.choice([1, 2, 5, 8]), rng.choice([64, 80, 128, 128])
    if op == "keep":
        return {"op": op, "requests": _log(rng, 1, 128), "ctx": _log(rng, 1, 600), "new": _log(rng, 2, 61),
                "layers": rng.choice([1, 2, 4]), "kv_heads": kv, "dim": dim, "block": block, "cache": cache}
    if op == "branch":
        return {"op": op, "requests": _log(rng, 1, 48), "children": rng.choice([1, 2, 3, 4]),
                "ctx": _log(rng, 1, 3000), "layers": rng.choice([1, 2, 4]), "kv_heads": kv, "dim": dim,
                "block": block, "cache": cache}
    requests = _log(rng, 1, 24)
    return {"op": op, "requests": requests, "ctx": min(16000, _log(rng, 16, 100000) // requests),
            "new": max(1, _log(rng, 8, 8000) // requests), "heads": kv * rng.choice([1, 3, 4, 8]), "kv_heads": kv,
            "dim": dim, "block": block, "cache": cache}


# ------------------------------------------------------------------ making the inputs
def _ladder(count, most, lowest=0):
    """`count` whole numbers from about lowest to `most`, the same for every seed."""
    return [lowest + int(round((most - lowest) * ((i + 1) / count) ** 1.5)) for i in range(count)]


def _lengths(case):
    """(tokens in the cache, new tokens) of the case's requests, before they are dealt out."""
    count = case["requests"]
    ctx = _ladder(count, case.get("ctx", 0), 1 if case["op"] == "branch" else 0)
    new = _ladder(count, case.get("new", 0), 1)
    return ctx, new[1::2] + new[::2]  # so that long contexts and many new tokens do not go together


def _requests(case, seed):
    ctx, new = _lengths(case)
    order = list(range(case["requests"]))
    random.Random(seed).shuffle(order)
    return np.array([ctx[i] for i in order], np.int32), np.array([new[i] for i in order], np.int32)


def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(g, shape, dtype, scale=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def _dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to("cuda")


def _tables(ctx, new, block, width, seed):
    """Distinct random pages for every request's tokens, -1 past them; (table, number of pages)."""
    pages = (ctx.astype(np.int64) + new + block - 1) // block
    total = int(pages.sum()) + 3
    ids = np.random.default_rng(seed).permutation(total)
    table = np.full((len(ctx), width), -1, np.int32)
    at = 0
    for b, p in enumerate(pages):
        table[b, :p] = ids[at:at + p]
        at += int(p)
    return table, total


def _cu(new):
    return np.concatenate([[0], np.cumsum(new)]).astype(np.int32)


def _slots(table, ctx, new, block):
    """Positions and slots of the new tokens."""
    pos = np.concatenate([np.arange(c, c + n) for c, n in zip(ctx, new)])
    row = np.repeat(np.arange(len(new)), new)
    return pos, table[row, pos // block].astype(np.int64) * block + pos % block


def _parents(case, new, seed):
    """Parents within each request's tree; row 0 is its only root.  A node has up to three
    children, in an order that has every parent before them."""
    rng = np.random.default_rng(seed)
    out = []
    for n in new:
        room, parents = [0] * 3, [-1]
        for i in range(1, int(n)):
            parents.append(room.pop(int(rng.integers(max(0, len(room) - 6), len(room)))) if case["tree"] else i - 1)
            room += [i] * 3
        out += parents[:int(n)]
    return np.array(out, np.int32)


def prepare(case, seed):
    g = _generator(seed)
    state = {"case": case, "ws": None, "out": None}
    return state | _prepare[case["op"]](case, seed, g)


def _prepare_rope(case, seed, g):
    ctx, new = _requests(case, seed)
    h, kv, d, block = case["heads"], case["kv_heads"], case["dim"], case["block"]
    dtype = _DTYPES[case["cache"]]
    # the pool has pages of the new tokens only: the ones before them are not looked at
    keep = np.minimum(ctx, ctx % block + 40)
    table, pages = _tables(keep, new, block, int((keep + new).max()) // block + 1, seed)
    pos, slots = _slots(table, keep, new, block)
    pos = pos + np.repeat(ctx - keep, new)
    slots[1::97] = -1  # rows of a padded batch that belong to no request
    pos[1::97] = -1
    qkv = _normal(g, (len(pos), (h + 2 * kv) * d), dtype if case["source"] == "same" else _DTYPES["f32"])
    split = qkv.view(len(pos), h + 2 * kv, d)
    gains = [1.0 + 0.2 * torch.randn(d, generator=g, device="cuda") for _ in range(2)]
    freqs = 500000.0 ** -(torch.arange(case["pairs"], device="cuda", dtype=torch.float64) / case["pairs"])
    return {"q": split[:, :h], "k": split[:, h:h + kv], "v": split[:, h + kv:], "slots": _dev(slots.astype(np.int32)),
            "positions": _dev(pos.astype(np.int32)), "freqs": freqs,
            "q_weight": gains[0] if case["norms"] else None, "k_weight": gains[1] if case["norms"] else None,
            "q_out": torch.zeros((len(pos), h, d), dtype=dtype, device="cuda"),
            "k_cache": _normal(g, (pages, kv, block, d), dtype), "v_cache": _normal(g, (pages, kv, d, block), dtype)}


# probabilities of a node's drafted children under the target, as trees meet them
_SHARES = (0.55, 0.2, 0.1)


def _prepare_verify(case, seed, g):
    _, new = _requests(case, seed)
    cu, vocab, count = _cu(new), case["vocab"], len(new)
    tokens = int(cu[-1])
    parents = _parents(case, new, seed)
    up = _dev(np.where(parents >= 0, parents + np.repeat(cu[:-1], new), -1)).long()
    logits = torch.randn((tokens, vocab), generator=g, device="cuda").mul_(2.0)
    u = torch.rand(tokens, generator=g, device="cuda")
    state = {"cu": _dev(cu), "parents": _dev(parents) if case["tree"] else None, "probs": None, "most": int(new.max()),
             "accept": u, "sample": torch.rand(count, generator=g, device="cuda"), "temperature": None}
    if case["probs"]:
        # a draft that is near the target, and its sample for each next token
        noise = torch.randn((tokens, vocab), generator=g, device="cuda")
        probs = torch.softmax((logits + noise.mul_(0.7)) * 1.2, 1)
        del noise
        pick = torch.rand(tokens, generator=g, device="cuda", dtype=torch.float64)[:, None]
        chosen = torch.searchsorted(torch.cumsum(probs, 1, dtype=torch.float64), pick)[:, 0].clamp(max=vocab - 1)
        state["probs"] = probs
    else:
        # the tree's children are the draft's best tokens; the target gives them their shares
        total = torch.logsumexp(logits, 1)
        order = np.zeros(len(parents), np.int64)  # which child of its parent a node is
        seen = {}
        for i, p in enumerate(up.tolist()):
            order[i] = seen.get(p, 0)
            seen[p] = order[i] + 1
        chosen = torch.randint(vocab, (tokens, 3), generator=g, device="cuda")
        rest = 1.0 - sum(_SHARES)
        for i, share in enumerate(_SHARES):
            at = chosen[:, i:i + 1]
            logits.scatter_(1, at, (total + math.log(share / rest))[:, None])
    mine = up.clamp(min=0)
    state["draft"] = (chosen[mine] if case["probs"] else chosen[mine, _dev(order).clamp(max=2)]).int()
    if case["greedy"]:
        # every third request takes the most likely token, the others have temperatures of their own
        t = 0.7 + 0.6 * torch.rand(count, generator=g, device="cuda")
        state["temperature"] = torch.where(torch.arange(count, device="cuda") % 3 == 0, torch.zeros_like(t), t)
    return state | {"logits": logits.to(_DTYPES[case["logits"]])}


def _kept(n):
    """How many of a request's n new tokens are kept."""
    return max(1, min(n, int(round(1.3 * n ** 0.5))))


def _prepare_keep(case, seed, g):
    ctx, new = _requests(case, seed)
    kv, d, block, layers = case["kv_heads"], case["dim"], case["block"], case["layers"]
    table, pages = _tables(ctx, new, block, int((ctx + new).max()) // block + 1, seed)
    _, slots = _slots(table, ctx, new, block)
    rng, kept = np.random.default_rng(seed + 1), np.array([_kept(int(n)) for n in new], np.int32)
    path = np.full(int(new.sum()), -1, np.int32)
    at = 0
    for n, k in zip(new, kept):
        # row 0, and an upward way through the later nodes of the tree
        later = np.arange(min(k, n - k + 1), n)
        path[at:at + k] = np.concatenate([[0], np.sort(rng.choice(later, k - 1, replace=False))]) if k > 1 else 0
        at += n
    dtype, head = _DTYPES[case["cache"]], int(new.sum()) + 5
    return {"path": _dev(path), "kept": _dev(kept), "ctx": _dev(ctx), "cu": _dev(_cu(new)),
            "slots": _dev(slots.astype(np.int32)), "table": _dev(table),
            "free": _dev(np.arange(head + 40, dtype=np.int32) + pages),
            "head": torch.tensor([head], dtype=torch.int32, device="cuda"), "lens": _dev(ctx),
            "counts": torch.zeros(2, dtype=torch.int32, device="cuda"),
            "k_cache": _normal(g, (layers, pages, kv, block, d), dtype),
            "v_cache": _normal(g, (layers, pages, kv, d, block), dtype)}


def _prepare_branch(case, seed, g):
    ctx, _ = _requests(case, seed)
    kv, d, block, layers, many = (case[x] for x in ("kv_heads", "dim", "block", "layers", "children"))
    count = len(ctx)
    own_table, pages = _tables(ctx, np.zeros_like(ctx), block, int(ctx.max()) // block + 9, seed)
    table = np.full((count * (1 + many), own_table.shape[1]), -1, np.int32)
    table[:count] = own_table
    forks, dtype = count * many, _DTYPES[case["cache"]]
    blocks = pages + forks + 3
    return {"src": _dev(np.repeat(np.arange(count), many).astype(np.int32)),
            "dst": _dev(np.arange(count, count + forks).astype(np.int32)),
            "lens": _dev(np.concatenate([ctx, np.zeros(forks, np.int32)])), "table": _dev(table),
            "free": _dev(np.concatenate([np.full(7, -1), np.arange(pages, blocks)]).astype(np.int32)),
            "head": torch.tensor([7], dtype=torch.int32, device="cuda"),
            "shares": torch.zeros(blocks, dtype=torch.int32, device="cuda"),
            "counts": torch.zeros(2, dtype=torch.int32, device="cuda"),
            "freed": torch.zeros(2, dtype=torch.int32, device="cuda"),
            "k_cache": _normal(g, (layers, blocks, kv, block, d), dtype),
            "v_cache": _normal(g, (layers, blocks, kv, d, block), dtype)}


def _prepare_chunk(case, seed, g):
    ctx, new = _requests(case, seed)
    h, kv, d, block = case["heads"], case["kv_heads"], case["dim"], case["block"]
    dtype = _DTYPES[case["cache"]]
    table, pages = _tables(ctx, new, block, int((ctx + new).max()) // block + 1, seed)
    cu = _cu(new)
    # queries and keys at the spread that gives a softmax a few dozen heavy keys
    return {"q": _normal(g, (int(cu[-1]), h, d), dtype, 1.4), "k_cache": _normal(g, (pages, kv, block, d), dtype, 1.4),
            "v_cache": _normal(g, (pages, kv, d, block), dtype), "table": _dev(table), "ctx": _dev(ctx),
            "cu": _dev(cu), "spans": [(int(c), int(n)) for c, n in zip(ctx, new)]}


_prepare = {"rope": _prepare_rope, "verify": _prepare_verify, "keep": _prepare_keep, "branch": _prepare_branch,
            "chunk": _prepare_chunk}


def run(state):
    return (_own if own else _plain)[state["case"]["op"]](state)


# ------------------------------------------------------------- the library's calls
def _own_rope(s):
    import decode_gemm_tile_amd as dgt
    q = dgt.dgt_rope_store(s["q"], s["k"], s["v"], s["positions"], s["slots"], s["freqs"], s["k_cache"], s["v_cache"],
                           q_weight=s["q_weight"], k_weight=s["k_weight"], interleaved=s["case"]["interleaved"],
                           q_out=s["q_out"])
    return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _own_verify(s):
    import decode_gemm_tile_amd as dgt
    if s["ws"] is None:  # made by the first pass and kept
        s["ws"] = dgt.alloc_workspace(dgt.dgt_verify_workspace(*s["logits"].shape, s["cu"].numel() - 1))
    v = s["out"] = dgt.dgt_verify(s["logits"], s["draft"], s["cu"], s["accept"], s["sample"], parents=s["parents"],
                                  draft_probs=s["probs"], temperature=s["temperature"], out=s["out"], ws=s["ws"])
    return {"path": v.path, "accepted": v.accepted, "next": v.next}


def _own_keep(s):
    import decode_gemm_tile_amd as dgt
    dgt.dgt_page_keep(s["kept"], s["ctx"], s["cu"], s["slots"], s["free"], s["head"], s["table"], s["k_cache"],
                      s["v_cache"], path=s["path"], lens=s["lens"], counts=s["counts"])
    return {x: s[x] for x in ("k_cache", "v_cache", "lens", "table", "free", "counts")}


def _own_branch(s):
    import decode_gemm_tile_amd as dgt
    if s["ws"] is None:  # made by the first pass and kept
        s["ws"] = dgt.alloc_workspace(dgt.dgt_page_free_workspace(s["shares"].numel()))
    dgt.dgt_page_fork(s["src"], s["dst"], s["lens"], s["free"], s["head"], s["table"], s["shares"], s["k_cache"],
                      s["v_cache"], counts=s["counts"])
    dgt.dgt_page_free(s["dst"], s["lens"], s["free"], s["counts"][:1], s["table"], s["shares"], s["case"]["block"],
                      counts=s["freed"], ws=s["ws"])
    return {x: s[x] for x in ("k_cache", "v_cache", "lens", "table", "free", "shares", "counts", "freed")}


def _own_chunk(s):
    import decode_gemm_tile_amd as dgt
    if s["ws"] is None:  # made by the first pass and kept
        s["ws"] = dgt.alloc_workspace(dgt.dgt_chunk_attention_workspace(
            s["q"].shape, s["k_cache"].shape[1], s["ctx"].numel()))
    return dgt.dgt_chunk_attention(s["q"], s["k_cache"], s["v_cache"], s["table"], s["ctx"], s["cu"], ws=s["ws"])


_own = {"rope": _own_rope, "verify": _own_verify, "keep": _own_keep, "branch": _own_branch, "chunk": _own_chunk}


# ------------------------------------------------------------------ the plain forms
def _plain_turn(x, weight, cos, sin, interleaved):
    x = x.float()
    if weight is not None:
        x = x * torch.rsqrt((x * x).mean(2, keepdim=True) + 1e-6) * weight
    pairs = cos.shape[2]
    if interleaved:
        a, b = x[:, :, 0:2 * pairs:2], x[:, :, 1:2 * pairs:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], 3).flatten(2)
    else:
        a, b = x[:, :, :pairs], x[:, :, pairs:2 * pairs]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], 2)
    return torch.cat([turned, x[:, :, 2 * pairs:]], 2)


def _plain_rope(s):
    block, dtype, interleaved = s["case"]["block"], s["k_cache"].dtype, s["case"]["interleaved"]
    live = s["positions"] >= 0
    angle = (s["positions"][live].double()[:, None] * s["freqs"])[:, None]
    cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
    s["q_out"][live] = _plain_turn(s["q"][live], s["q_weight"], cos, sin, interleaved).to(dtype)
    keys = _plain_turn(s["k"][live], s["k_weight"], cos, sin, interleaved).to(dtype)
    slot = s["slots"][live].long()
    s["k_cache"][slot // block, :, slot % block] = keys
    s["v_cache"][slot // block, :, :, slot % block] = s["v"][live].to(dtype)
    return {"q": s["q_out"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _plain_verify(s):
    """All requests side by side, the nodes of their trees one after another: a node is
    looked at if its parent is the path's end."""
    cu, logits, vocab = s["cu"].long(), s["logits"], s["case"]["vocab"]
    count, tokens = cu.numel() - 1, logits.shape[0]
    first, new = cu[:-1], cu[1:] - cu[:-1]
    every = torch.arange(count, device=cu.device)
    owner = torch.searchsorted(cu, torch.arange(tokens, device=cu.device), right=True) - 1
    heat = s["temperature"] if s["temperature"] is not None else torch.ones(count, device=cu.device)
    greedy = heat <= 0
    # sums over a vocabulary and the border that a uniform number falls behind need 64 bits
    p = logits.double()
    best = torch.where(p == p.amax(1, keepdim=True), torch.arange(vocab, device=cu.device), vocab).amin(1)
    p = torch.exp((p - p.amax(1, keepdim=True)) / torch.where(greedy, 1.0, heat)[owner].double()[:, None])
    p /= p.sum(1, keepdim=True)
    left = torch.ones(count, dtype=torch.float64, device=cu.device)  # of the mass at the path's end
    refused = torch.zeros(count, dtype=torch.bool, device=cu.device)
    end, length = torch.zeros_like(every), (new > 0).long()
    path = torch.full((tokens + 1,), -1, dtype=torch.int64, device=cu.device)
    path[torch.where(new > 0, first, tokens)] = 0
    for j in range(1, s["most"]):
        row = (first + j).clamp(max=tokens - 1)
        up = s["parents"][row] if s["parents"] is not None else j - 1
        looked = (j < new) & (up == end)
        at, x = (first + end).clamp(max=tokens - 1), s["draft"][row].long()
        mine = p[at, x]
        q = s["probs"][at, x].double() if s["probs"] is not None else 1.0
        taken = looked & torch.where(greedy, x == best[at], s["accept"][row].double() * left * q < mine)
        lost = looked & ~taken
        refused = (refused | lost) & ~taken
        if s["probs"] is None:
            left = torch.where(lost, left - mine, torch.where(taken, 1.0, left))
            p[at, x] = torch.where(lost, 0.0, mine)
        end = torch.where(taken, j, end)
        path[torch.where(taken, first + length, tokens)] = j
        length = length + taken
    at = (first + end).clamp(max=tokens - 1)
    rest = p[at]
    if s["probs"] is not None:
        rest = torch.where(refused[:, None], (rest - s["probs"][at].double()).clamp_(min=0), rest)
    run_sum = torch.cumsum(rest, 1)
    border = s["sample"].double()[:, None] * run_sum[:, -1:]
    token = torch.where(greedy, best[at], (run_sum <= border).sum(1).clamp(max=vocab - 1))
    return {"path": path[:tokens].int(), "accepted": length.int(), "next": torch.where(new > 0, token, -1).int()}


def _plain_keep(s):
    cu, block, blocks = s["cu"].long(), s["case"]["block"], s["k_cache"].shape[1]
    count, tokens = cu.numel() - 1, s["slots"].numel()
    t = torch.arange(tokens, device=cu.device)
    row = torch.searchsorted(cu, t, right=True) - 1
    at = t - cu[row]
    moved = (at < s["kept"][row]) & (s["path"] != at)
    src = s["slots"][(cu[row] + s["path"])[moved]].long()
    dst = s["slots"][moved].long()
    for k, v in zip(s["k_cache"], s["v_cache"]):
        k[dst // block, :, dst % block] = k[src // block, :, src % block]
        v[dst // block, :, :, dst % block] = v[src // block, :, :, src % block]
    torch.add(s["ctx"], s["kept"], out=s["lens"])
    pages = (s["lens"] + block - 1) // block
    after = (s["ctx"] + cu[1:] - cu[:-1] + block - 1) // block
    # pages that begin past the kept tokens: the new token that lies first in each names it
    pos = s["ctx"][row] + at
    page = pos // block
    gone = (page >= pages[row]) & ((pos % block == 0) | (at == 0))
    ids = s["slots"][gone] // block
    number = (after - pages).clamp(min=0).sum(dtype=torch.int32)
    head = s["head"] - number
    s["free"][head + torch.arange(ids.numel(), device=cu.device)] = ids
    s["table"][row[gone], page[gone]] = -1
    s["counts"].copy_(torch.cat([head, number[None]]))
    return {x: s[x] for x in ("k_cache", "v_cache", "lens", "table", "free", "counts")}


def _plain_branch(s):
    block, src, dst, table, shares = s["case"]["block"], s["src"].long(), s["dst"].long(), s["table"], s["shares"]
    # fork: full pages are shared, a part of one is copied into a page of the free list
    lens = s["lens"][src]
    full, part = lens // block, lens % block
    need = part > 0
    fresh = s["free"][(s["head"] + torch.cumsum(need, 0) - 1).clamp(max=s["free"].numel() - 1)]
    col = torch.arange(table.shape[1], device=src.device)
    rows = torch.where(col < full[:, None], table[src], -1)
    rows = torch.where((col == full[:, None]) & need[:, None], fresh[:, None], rows)
    table[dst] = torch.where(rows >= 0, rows, table[dst])
    held = rows[(col < full[:, None]) & (rows >= 0)].long()
    shares += torch.bincount(held, minlength=shares.numel()).int()
    a = table[src, full.clamp(max=table.shape[1] - 1)][need].long()
    b, n = fresh[need].long(), part[need]
    cell = torch.arange(block, device=src.device) < n[:, None]
    for k, v in zip(s["k_cache"], s["v_cache"]):
        k[b] = torch.where(cell[:, None, :, None], k[a], k[b])
        v[b] = torch.where(cell[:, None, None, :], v[a], v[b])
    s["lens"][dst] = lens
    s["counts"].copy_(torch.stack([s["head"][0] + need.sum(), torch.zeros_like(need.sum())]))
    # free: the last holder of a page returns it, in the order of the pages' numbers
    pages = (s["lens"][dst] + block - 1) // block
    mine = (col < pages[:, None]) & (table[dst] >= 0)
    shares -= torch.bincount(table[dst][mine].long(), minlength=shares.numel()).int()
    ids = torch.nonzero(shares < 0)[:, 0].int()
    shares.clamp_(min=0)
    table[dst] = torch.where(mine, -1, table[dst])
    s["lens"][dst] = 0
    head = s["counts"][0] - ids.numel()
    s["free"][head + torch.arange(ids.numel(), device=src.device)] = ids
    s["freed"].copy_(torch.stack([head, torch.full_like(head, ids.numel())]))
    return {x: s[x] for x in ("k_cache", "v_cache", "lens", "table", "free", "shares", "counts", "freed")}


def _plain_chunk(s):
    h, kv, d, block = (s["case"][x] for x in ("heads", "kv_heads", "dim", "block"))
    group, at, outs = h // kv, 0, torch.empty_like(s["q"])
    for b, (c, n) in enumerate(s["spans"]):
        if n == 0:
            continue
        ids = s["table"][b, :-(-(c + n) // block)]
        seen = torch.arange(c + n, device=ids.device) <= c + torch.arange(n, device=ids.device)[:, None]
        for x in range(kv):
            keys = s["k_cache"][ids, x].reshape(-1, d)[:c + n].float()
            values = s["v_cache"][ids, x].transpose(1, 2).reshape(-1, d)[:c + n].float()
            q = s["q"][at:at + n, x * group:(x + 1) * group].transpose(0, 1).float()
            scores = torch.matmul(q, keys.t()).mul_(d ** -0.5).masked_fill_(~seen, -math.inf)
            scores = scores.sub_(scores.amax(2, keepdim=True)).exp_()
            total = scores.sum(2, keepdim=True)
            outs[at:at + n, x * group:(x + 1) * group] = (torch.matmul(scores, values) / total).transpose(0, 1).to(outs.dtype)
            del scores
        at += n
    return outs


_plain = {"rope": _plain_rope, "verify": _plain_verify, "keep": _plain_keep, "branch": _plain_branch,
          "chunk": _plain_chunk}


# -------------------------------------------------------------------------- the work
def work(case):
    ctx, new = _lengths(case)
    tokens, op = sum(new), case["op"]
    if op == "rope":
        size = 2 if case["source"] == "same" else 4
        values = tokens * (case["heads"] + 2 * case["kv_heads"]) * case["dim"]
        turned = tokens * (case["heads"] + case["kv_heads"]) * case["dim"]
        return {"bytes": values * (size + 2) + 8 * tokens, "flops": turned * (8 if case["norms"] else 3)}
    if op == "verify":
        # rows on the accepted path: of a chain about three of four drafted tokens are taken;
        # a tree's three children hold 85% of the target, and its path ends at a leaf
        rate, size = (0.75, 4 if case["logits"] == "f32" else 2)
        depth = [math.log2(1 + n) if case["tree"] else n for n in new]
        rows = sum((1 - rate ** n) / (1 - rate) for n in depth)
        ends = sum(1 - rate ** n for n in depth) if case["probs"] else 0
        return {"bytes": case["vocab"] * (rows * size + 4 * ends) + 12 * tokens, "flops": 4 * rows * case["vocab"]}
    if op == "chunk":
        h, kv, d = case["heads"], case["kv_heads"], case["dim"]
        cached = sum(c + n for c, n in zip(ctx, new)) * kv * d * 2 * 2
        return {"bytes": cached + 2 * tokens * h * d * 2 + sum((c + n) // case["block"] + 1 for c, n in zip(ctx, new)) * 4,
                "flops": sum(4 * n * (c + (n + 1) / 2) * h * d for c, n in zip(ctx, new))}
    row = case["layers"] * case["kv_heads"] * case["dim"] * 2 * 2  # of a token, keys and values
    if op == "keep":
        moved = sum(_kept(n) - 1 for n in new)
        return {"bytes": 2 * moved * row + 4 * tokens + 20 * case["requests"], "flops": 2 * tokens}
    many, block = case["children"], case["block"]
    copied = many * sum(c % block for c in ctx)
    entries = many * sum(-(-c // block) for c in ctx)
    return {"bytes": 2 * copied * row + 16 * entries, "flops": 2 * entries}


# ------------------------------------------------- the definitions, in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return {"rope": _exact_rope, "verify": _exact_verify, "keep": _exact_keep, "branch": _exact_branch,
            "chunk": _exact_chunk}[case["op"]](s)


def _exact_rope(s):
    case, positions, slots = s["case"], s["positions"].cpu().numpy(), s["slots"].cpu().tolist()
    d, pairs, block = case["dim"], case["pairs"], case["block"]
    angle = positions.astype(np.float64)[:, None] * s["freqs"].cpu().numpy()
    turn = torch.from_numpy(np.exp(1j * angle)).to("cuda")[:, None]

    def turned(x, weight):
        x = x.double()
        if weight is not None:
            x = weight.double() * x / torch.sqrt(x.square().sum(2, keepdim=True) / d + 1e-6)
        x = x.clone()
        i = torch.arange(pairs, device="cuda")
        lo, hi = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + pairs)
        z = torch.complex(x[:, :, lo], x[:, :, hi]) * turn
        x[:, :, lo], x[:, :, hi] = z.real, z.imag
        return x

    keep = [t for t, slot in enumerate(slots) if slot >= 0]
    rows = torch.tensor(keep, device="cuda")
    page = torch.tensor([slots[t] // block for t in keep], device="cuda")
    cell = torch.tensor([slots[t] % block for t in keep], device="cuda")
    outs = {"q": s["q_out"].double(), "k_cache": s["k_cache"].double(), "v_cache": s["v_cache"].double()}
    live = torch.from_numpy(np.nonzero(positions >= 0)[0]).to("cuda")
    outs["q"][live] = turned(s["q"], s["q_weight"])[live]
    outs["k_cache"].transpose(1, 2)[page, cell] = turned(s["k"], s["k_weight"])[rows]
    outs["v_cache"].permute(0, 3, 1, 2)[page, cell] = s["v"].double()[rows]
    return outs


def _exact_verify(s):
    cu, draft = s["cu"].cpu().tolist(), s["draft"].cpu().tolist()
    accept, sample = s["accept"].cpu().tolist(), s["sample"].cpu().tolist()
    heat = s["temperature"].cpu().tolist() if s["temperature"] is not None else None
    parents = s["parents"].cpu().tolist() if s["parents"] is not None else None
    path, accepted, following = np.full(len(draft), -1, np.int32), [], []
    for b in range(len(cu) - 1):
        start, n = cu[b], cu[b + 1] - cu[b]
        t = 1.0 if heat is None else heat[b]
        way = [0] if n else []
        token = -1
        while way:
            row = s["logits"][start + way[-1]].double()
            children = [j for j in range(way[-1] + 1, n) if (parents[start + j] if parents else j - 1) == way[-1]]
            go = None
            if t <= 0:
                token = int(torch.nonzero(row == row.max())[0, 0])
                go = next((j for j in children if draft[start + j] == token), None)
            else:
                p = torch.softmax(row / t, 0)
                for j in children:
                    x = draft[start + j]
                    q = float(s["probs"][start + way[-1], x]) if s["probs"] is not None else 1.0
                    if accept[start + j] * float(p.sum()) * q < float(p[x]):
                        go = j
                        break
                    if s["probs"] is not None:
                        p = (p - s["probs"][start + way[-1]].double()).clamp(min=0)
                    else:
                        p[x] = 0.0
                if go is None:
                    total = torch.cumsum(p, 0)
                    token = int(torch.searchsorted(total, total[-1:] * sample[b], right=True)[0].clamp(max=len(p) - 1))
            if go is None:
                break
            way.append(go)
        path[start:start + len(way)] = way
        accepted.append(len(way))
        following.append(token)
    return {"path": path, "accepted": np.array(accepted, np.int32), "next": np.array(following, np.int32)}


def _exact_keep(s):
    ctx, kept, cu, slots, path = (s[x].cpu().tolist() for x in ("ctx", "kept", "cu", "slots", "path"))
    block, table, free = s["case"]["block"], s["table"].cpu().numpy().copy(), s["free"].cpu().numpy().copy()
    src, dst, gone, lens = [], [], [], []
    for b, c in enumerate(ctx):
        n = cu[b + 1] - cu[b]
        lens.append(c + kept[b])
        for j in range(kept[b]):
            src.append(slots[cu[b] + path[cu[b] + j]])
            dst.append(slots[cu[b] + j])
        for p in range(-(-lens[b] // block), -(-(c + n) // block)):
            gone.append(int(table[b, p]))
            table[b, p] = -1
    head = int(s["head"].item()) - len(gone)
    free[head:head + len(gone)] = gone
    src, dst = torch.tensor(src, device="cuda"), torch.tensor(dst, device="cuda")
    k, v = s["k_cache"].double().transpose(2, 3).contiguous(), s["v_cache"].double().permute(0, 1, 4, 2, 3).contiguous()
    for x in (k, v):
        x.flatten(1, 2)[:, dst] = x.flatten(1, 2)[:, src]
    return {"k_cache": k.transpose(2, 3), "v_cache": v.permute(0, 1, 3, 4, 2), "lens": np.array(lens, np.int32),
            "table": table, "free": free, "counts": np.array([head, len(gone)], np.int32)}


def _exact_branch(s):
    src, dst, lens = (s[x].cpu().tolist() for x in ("src", "dst", "lens"))
    block, table, free = s["case"]["block"], s["table"].cpu().numpy().copy(), s["free"].cpu().numpy().copy()
    head, held, fresh = int(s["head"].item()), {}, []
    k, v = s["k_cache"].double(), s["v_cache"].double()
    for a, b in zip(src, dst):
        rows = table[a, :lens[a] // block].tolist()
        for p in rows:
            held[p] = held.get(p, 0) + 1
        n = lens[a] % block
        if n:
            page, old = int(free[head + len(fresh)]), int(table[a, lens[a] // block])
            fresh.append(page)
            k[:, page, :, :n] = k[:, old, :, :n]
            v[:, page, :, :, :n] = v[:, old, :, :, :n]
    # the children's shares of full pages end with them; their own pages go back, by number
    fresh.sort()
    free[head:head + len(fresh)] = fresh
    return {"k_cache": k, "v_cache": v, "lens": np.array(lens, np.int32), "table": table, "free": free,
            "shares": np.zeros(s["shares"].numel(), np.int32),
            "counts": np.array([head + len(fresh), 0], np.int32), "freed": np.array([head, len(fresh)], np.int32)}


def _exact_chunk(s):
    d, block, group = s["case"]["dim"], s["case"]["block"], s["case"]["heads"] // s["case"]["kv_heads"]
    if sum(n * (c + n) for c, n in s["spans"]) * s["case"]["heads"] > 2 ** 33:
        return None
    outs = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    start = 0
    for b, (c, n) in enumerate(s["spans"]):
        ids = s["table"][b, :-(-(c + n) // block)].long()
        hidden = torch.ones((n, c + n), dtype=torch.bool, device="cuda").triu(c + 1)
        for x in range(s["q"].shape[1]):
            keys = s["k_cache"][ids, x // group].reshape(-1, d)[:c + n].double()
            values = s["v_cache"][ids, x // group].transpose(1, 2).reshape(-1, d)[:c + n].double()
            z = s["q"][start:start + n, x].double() @ keys.t() / math.sqrt(d)
            z[hidden] = -math.inf
            outs[start:start + n, x] = torch.exp(z - torch.logsumexp(z, 1, keepdim=True)) @ values
        start += n
    return outs
