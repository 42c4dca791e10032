"""Measured cases of the serving operators: the page plan of a step, the store of
new keys and values, attention for trees of drafted tokens over a paged cache, and
the low-rank adapters of many requests beside a shared projection.

``run`` computes a case either with the library's kernels (``own = True``) or in a
plain form of elementary torch operations in 32 bits (``own = False``); both take
the state that ``prepare`` makes.  ``exact`` computes the same outputs from the
definitions in 64 bits.

Shapes.  A request b holds ctx[b] tokens in the cache and brings new[b] tokens to
the step; the new tokens of all requests lie one after another in T rows.  Key
pages are [blocks, heads, block, dim]; value pages are transposed,
[blocks, heads, dim, block].  Lengths form a ladder from short to the stated
maximum, dealt to the requests in an order drawn from the seed, so a case's work
is the same for every seed.
"""

import math
import random

import numpy as np
import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def listed():
    return [
        # One step of a small decoding batch: every request brings one token; latency only.
        {"name": "plan_tokens", "op": "plan", "requests": 8, "ctx": 900, "new": 1, "tree": False,
         "block": 16, "width": 64},
        # A large batch that verifies trees of up to 61 drafted tokens each: tables, slots,
        # positions by depth and ancestor masks.
        {"name": "plan_trees", "op": "plan", "requests": 509, "ctx": 32000, "new": 61, "tree": True,
         "block": 16, "width": 2048},
        # The keys and values of a small decoding step, read out of the fp32 rows that the
        # fused qkv projection writes.
        {"name": "store_tokens", "op": "store", "requests": 5, "ctx": 700, "new": 1, "heads": 32,
         "kv_heads": 8, "dim": 128, "block": 16, "source": "f32", "cache": "bf16"},
        # Prompts of uneven lengths going into the cache in one step.
        {"name": "store_prompts", "op": "store", "requests": 7, "ctx": 500, "new": 2047, "heads": 32,
         "kv_heads": 8, "dim": 128, "block": 16, "source": "f32", "cache": "bf16"},
        # One user, one token, a short context: the latency of a decoding step.
        {"name": "attn_token", "op": "attention", "requests": 1, "ctx": 1000, "new": 1, "tree": False,
         "heads": 32, "kv_heads": 8, "dim": 128, "block": 16, "cache": "bf16"},
        # A decoding batch with ragged contexts, one token each: the cache is read once.
        {"name": "attn_batch", "op": "attention", "requests": 96, "ctx": 8100, "new": 1, "tree": False,
         "heads": 32, "kv_heads": 8, "dim": 128, "block": 16, "cache": "bf16"},
        # Trees of up to 27 drafted tokens for a medium batch.
        {"name": "attn_trees", "op": "attention", "requests": 16, "ctx": 4090, "new": 27, "tree": True,
         "heads": 32, "kv_heads": 8, "dim": 128, "block": 16, "cache": "bf16"},
        # Long documents on a model with 16 query heads to a key head, trees of up to 29.
        {"name": "attn_long", "op": "attention", "requests": 4, "ctx": 131000, "new": 29, "tree": True,
         "heads": 128, "kv_heads": 8, "dim": 128, "block": 64, "cache": "bf16"},
        # Half precision, one key head to each query head, narrow heads, a drafted chain.
        {"name": "attn_chain", "op": "attention", "requests": 33, "ctx": 1531, "new": 7, "tree": False,
         "heads": 12, "kv_heads": 12, "dim": 64, "block": 32, "cache": "f16"},
        # One token through one adapter beside a 4096 x 4096 projection: latency.
        {"name": "lora_token", "op": "lora", "requests": 1, "new": 1, "adapters": 1, "rank": 16,
         "n": 4096, "k": 4096},
        # 64 users, each with an adapter of their own, one token each, beside the
        # 405B-scale FFN projection: the adapters are read once.
        {"name": "lora_users", "op": "lora", "requests": 64, "new": 1, "adapters": 56, "rank": 16,
         "n": 53248, "k": 16384},
        # Prompts of uneven lengths through wider adapters beside the 14336 x 4096 projection.
        {"name": "lora_prompts", "op": "lora", "requests": 6, "new": 701, "adapters": 4, "rank": 64,
         "n": 14336, "k": 4096},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["plan", "store", "attention", "attention", "lora"])
    if op == "plan":
        tree = rng.random() < 0.5
        block = rng.choice([16, 32, 64])
        ctx, new = _log(rng, 1, 32000), _log(rng, 1, 61)
        return {"op": op, "requests": _log(rng, 1, 509), "ctx": ctx, "new": new, "tree": tree,
                "block": block, "width": (ctx + new) // block + 1 + rng.randrange(40)}
    if op == "store":
        kv, requests = rng.choice([1, 2, 3, 8]), _log(rng, 1, 64)
        return {"op": op, "requests": requests, "ctx": _log(rng, 1, 900),
                "new": max(1, min(2047, _log(rng, 1, 8000) // requests)), "heads": kv * rng.choice([1, 4]),
                "kv_heads": kv, "dim": rng.choice([64, 80, 128]), "block": rng.choice([16, 32, 64]),
                "source": rng.choice(["f32", "same"]), "cache": rng.choice(["bf16", "f16"])}
    if op == "attention":
        kv, tree, requests = rng.choice([1, 2, 5, 8]), rng.random() < 0.6, _log(rng, 1, 96)
        ctx = max(1, min(131000, _log(rng, 16, 500000) // requests))
        return {"op": op, "requests": requests, "ctx": ctx, "new": rng.choice([1, 1, 2, 5, 8, 13, 27, 61]),
                "tree": tree, "heads": kv * rng.choice([1, 3, 4, 8]), "kv_heads": kv,
                "dim": rng.choice([64, 80, 128, 128]), "block": rng.choice([16, 32, 64]),
                "cache": rng.choice(["bf16", "bf16", "f16"])}
    n, k = rng.choice([(4096, 4096), (14336, 4096), (8192, 8192), (1024, 1024), (4096, 14336)])
    requests = _log(rng, 1, 64)
    return {"op": op, "requests": requests, "new": max(1, _log(rng, 1, 4000) // requests),
            "adapters": rng.randint(1, requests), "rank": rng.choice([8, 16, 24, 32, 64]), "n": n, "k": k}


def _ladder(count, most, lowest=0):
    """`count` whole numbers from about lowest to `most`, the same for every seed."""
    return [lowest + int(round((most - lowest) * ((i + 1) / count) ** 1.5)) for i in range(count)]


def _lengths(case):
    """(tokens in the cache, new tokens) of the case's requests, before they are dealt out."""
    count = case["requests"]
    ctx = _ladder(count, case.get("ctx", 0))
    new = _ladder(count, case["new"], 1)
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


def _tree(new, seed):
    """Parents within each request's tree (-1: the tree hangs off the cached context), in
    an order that has every parent before its children; a random recursive tree."""
    rng = np.random.default_rng(seed)
    parts = [np.concatenate([[-1], (rng.random(n - 1) * np.arange(1, n)).astype(np.int64)])[:n] for n in new]
    return np.concatenate(parts).astype(np.int32)


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


def _words(case):
    return (case["new"] + 63) // 64


def _ancestors(parents, cu, words):
    """Rows of bits: bit j of token i is set if j is i or one of its ancestors."""
    rows = np.zeros((len(parents), words), np.uint64)
    for b in range(len(cu) - 1):
        s = int(cu[b])
        for i in range(int(cu[b + 1]) - s):
            if parents[s + i] >= 0:
                rows[s + i] = rows[s + int(parents[s + i])]
            rows[s + i, i // 64] |= np.uint64(1) << np.uint64(i % 64)
    return rows.view(np.int64)


def prepare(case, seed):
    g = _generator(seed)
    state = {"case": case}
    if case["op"] == "plan":
        ctx, new = _requests(case, seed)
        block, width = case["block"], case["width"]
        total = int(new.sum())
        table, pages = _tables(ctx, np.zeros_like(new), block, width, seed)
        extra = int(((ctx + new + block - 1) // block - (ctx + block - 1) // block).sum())
        # some room is left in the free list, and some of it was taken by earlier steps
        free = np.random.default_rng(seed + 1).permutation(extra + 40) + pages
        state |= {"ctx": _dev(ctx), "new": _dev(new), "free": _dev(free.astype(np.int32)),
                  "head": torch.tensor([7], dtype=torch.int32, device="cuda"), "table": _dev(table),
                  "blocks": pages + extra + 40, "tokens": total, "parents": None, "words": 0, "out": None}
        if case["tree"]:
            state |= {"parents": _dev(_tree(new, seed)), "words": _words(case)}
        return state
    if case["op"] == "store":
        ctx, new = _requests(case, seed)
        h, kv, d, block = case["heads"], case["kv_heads"], case["dim"], case["block"]
        dtype = _DTYPES[case["cache"]]
        width = int((ctx + new).max()) // block + 1
        table, pages = _tables(ctx, new, block, width, seed)
        pos = np.concatenate([np.arange(c, c + n) for c, n in zip(ctx, new)])
        row = np.repeat(np.arange(len(new)), new)
        slots = table[row, pos // block].astype(np.int64) * block + pos % block
        slots[1::97] = -1  # rows of a padded batch that belong to no request
        qkv = _normal(g, (len(pos), (h + 2 * kv) * d), dtype if case["source"] == "same" else _DTYPES["f32"])
        split = qkv.view(len(pos), h + 2 * kv, d)
        state |= {"k": split[:, h:h + kv], "v": split[:, h + kv:], "slots": _dev(slots.astype(np.int32)),
                  "k_cache": _normal(g, (pages, kv, block, d), dtype),
                  "v_cache": _normal(g, (pages, kv, d, block), dtype)}
        return state
    if case["op"] == "attention":
        ctx, new = _requests(case, seed)
        h, kv, d, block = case["heads"], case["kv_heads"], case["dim"], case["block"]
        dtype = _DTYPES[case["cache"]]
        width = int((ctx + new).max()) // block + 1
        table, pages = _tables(ctx, new, block, width, seed)
        cu = _cu(new)
        # queries and keys at the spread that gives a softmax a few dozen heavy keys
        state |= {"q": _normal(g, (int(cu[-1]), h, d), dtype, 1.4),
                  "k_cache": _normal(g, (pages, kv, block, d), dtype, 1.4),
                  "v_cache": _normal(g, (pages, kv, d, block), dtype),
                  "table": _dev(table), "ctx": _dev(ctx), "cu": _dev(cu), "mask": None, "ws": None,
                  "most": int(new.max()), "longest": int((ctx + new).max())}
        if case["tree"]:
            state["mask"] = _dev(_ancestors(_tree(new, seed), cu, _words(case)))
        return state
    _, new = _requests(case, seed)
    n, k, r, count = case["n"], case["k"], case["rank"], case["adapters"]
    cu = _cu(new)
    # one request in eight (of several) uses no adapter; the others share them in turn
    ids = [-1 if b % 8 == 7 else b % count for b in range(len(new))]
    random.Random(seed + 1).shuffle(ids)
    state |= {"x": _normal(g, (int(cu[-1]), k), torch.bfloat16), "y": _normal(g, (int(cu[-1]), n), torch.float32),
              "a": _normal(g, (count, r, k), torch.bfloat16, k ** -0.5),
              "b": _normal(g, (count, n, r), torch.bfloat16, 0.3 * r ** -0.5),
              "scaling": 1.0 + torch.rand(count, generator=g, device="cuda"),
              "adapters": _dev(np.array(ids, np.int32)), "cu": _dev(cu), "ws": None}
    state["out"] = torch.empty_like(state["y"])
    return state


def run(state):
    return (_own if own else _plain)[state["case"]["op"]](state)


# ------------------------------------------------------------- the library's calls
def _own_plan(s):
    import decode_gemm_tile_amd as dgt
    p = s["out"] = dgt.dgt_page_plan(s["ctx"], s["new"], s["free"], s["head"], s["table"], s["case"]["block"],
                                     s["blocks"], s["tokens"], parents=s["parents"], mask_words=s["words"],
                                     out=s["out"])
    outs = {"table": s["table"], "cu": p.cu, "slots": p.slots, "positions": p.positions, "counts": p.counts}
    return outs | ({"mask": p.mask} if s["parents"] is not None else {})


def _own_store(s):
    import decode_gemm_tile_amd as dgt
    dgt.dgt_kv_store(s["k"], s["v"], s["slots"], s["k_cache"], s["v_cache"])
    return {"k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _own_attention(s):
    import decode_gemm_tile_amd as dgt
    if s["ws"] is None:  # made by the first pass and kept
        s["ws"] = dgt.alloc_workspace(dgt.dgt_tree_attention_workspace(
            s["q"].shape, s["k_cache"].shape[1], s["ctx"].numel()))
    return dgt.dgt_tree_attention(s["q"], s["k_cache"], s["v_cache"], s["table"], s["ctx"], s["cu"],
                                  mask=s["mask"], ws=s["ws"])


def _own_lora(s):
    import decode_gemm_tile_amd as dgt
    if s["ws"] is None:  # made by the first pass and kept
        s["ws"] = dgt.alloc_workspace(dgt.dgt_lora_workspace(
            s["x"].shape[0], s["cu"].numel() - 1, s["y"].shape[1], s["x"].shape[1], s["a"].shape[1]))
    return dgt.dgt_lora_add(s["y"], s["x"], s["a"], s["b"], s["scaling"], s["adapters"], s["cu"],
                            out=s["out"], ws=s["ws"])


_own = {"plan": _own_plan, "store": _own_store, "attention": _own_attention, "lora": _own_lora}


# ------------------------------------------------------------------ the plain forms
def _cu_of(new):
    return torch.nn.functional.pad(torch.cumsum(new, 0, dtype=torch.int32), (1, 0))


def _plain_plan(s):
    ctx, new, table, block = s["ctx"], s["new"], s["table"], s["case"]["block"]
    count, width, tokens = ctx.numel(), table.shape[1], s["tokens"]
    have = (ctx + block - 1) // block
    after = (ctx + new + block - 1) // block
    need = torch.where(after > width, 0, after - have)
    cu = _cu_of(new)
    end = s["head"] + torch.cumsum(need, 0, dtype=torch.int32)
    fits = (after <= width) & (cu[1:] <= tokens) & ((need == 0) | (end <= s["free"].numel()))
    t = torch.arange(tokens, dtype=torch.int32, device=cu.device)
    row = torch.searchsorted(cu, t, right=True).sub(1).clamp(max=count - 1)
    at = t - cu[row]
    live = (t < cu[-1]) & fits[row]
    pos = ctx[row] + at
    page = (pos // block).clamp(max=width - 1)
    fresh = (end - need)[row] + page - have[row]
    ids = torch.where(page >= have[row], s["free"][fresh.clamp(0, s["free"].numel() - 1)], table[row, page])
    slots = torch.where(live & (ids >= 0) & (ids < s["blocks"]), ids * block + pos % block, -1)
    taken = live & (page >= have[row])
    table[row[taken], page[taken]] = ids[taken]
    depth, outs = at, {}
    if s["parents"] is not None:
        own_bit = torch.arange(s["words"], device=cu.device) == (at // 64)[:, None]
        mask = torch.where(own_bit, torch.ones_like(at, dtype=torch.int64).bitwise_left_shift(at % 64)[:, None], 0)
        up = torch.where(s["parents"] >= 0, s["parents"] + cu[row], -1)
        depth = (up >= 0).int()
        # each round doubles the number of ancestors that a row has gathered
        for _ in range(max(1, (s["case"]["new"] - 1).bit_length())):
            has, to = up >= 0, up.clamp(min=0)
            mask = torch.where(has[:, None], mask | mask[to], mask)
            depth = torch.where(has, depth + depth[to], depth)
            up = torch.where(has, up[to], -1)
        outs["mask"] = torch.where((t < cu[-1])[:, None], mask, 0)
    positions = torch.where(t < cu[-1], ctx[row] + depth, -1)
    head = s["head"] + torch.where(fits, need, 0).sum(dtype=torch.int32)
    counts = torch.cat([cu[-1:], head, (~fits).sum(dtype=torch.int32)[None]])
    return {"table": table, "cu": cu, "slots": slots, "positions": positions, "counts": counts} | outs


def _plain_store(s):
    block = s["case"]["block"]
    valid = s["slots"] >= 0
    slot = s["slots"][valid].long()
    s["k_cache"][slot // block, :, slot % block] = s["k"][valid].to(s["k_cache"].dtype)
    s["v_cache"][slot // block, :, :, slot % block] = s["v"][valid].to(s["v_cache"].dtype)
    return {"k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _plain_attention(s):
    q, ctx, cu = s["q"], s["ctx"], s["cu"]
    h, kv, d, block = (s["case"][x] for x in ("heads", "kv_heads", "dim", "block"))
    count, most, pages = ctx.numel(), s["most"], (s["longest"] + block - 1) // block
    new = cu[1:] - cu[:-1]
    ids = s["table"][:, :pages].clamp(min=0)
    keys = s["k_cache"][ids].permute(0, 2, 1, 3, 4).reshape(count, kv, pages * block, d).float()
    at = torch.arange(most, device=q.device)
    rows = (cu[:-1, None] + at).clamp(max=q.shape[0] - 1)
    qs = q[rows].float().view(count, most, kv, h // kv, d).permute(0, 2, 1, 3, 4).reshape(count, kv, -1, d)
    scores = torch.matmul(qs, keys.transpose(2, 3)) * d ** -0.5
    del keys
    j = torch.arange(pages * block, device=q.device) - ctx[:, None]
    if s["mask"] is None:
        seen = j[:, None] <= at[:, None]
    else:
        word = s["mask"][rows][:, :, :, None].expand(-1, -1, -1, 64)
        bits = (word >> torch.arange(64, device=q.device)).bitwise_and(1).reshape(count, most, -1)
        pick = j.clamp(0, bits.shape[2] - 1)[:, None].expand(-1, most, -1)
        seen = (j < 0)[:, None] | (bits.gather(2, pick) != 0)
    seen = seen & (j < new[:, None])[:, None]
    seen = seen[:, None, :, None].expand(-1, 1, -1, h // kv, -1).reshape(count, 1, -1, pages * block)
    scores = scores.masked_fill_(~seen, -math.inf)
    top = scores.amax(3, keepdim=True)
    scores = scores.sub_(torch.where(top == -math.inf, 0.0, top)).exp_()
    total = scores.sum(3, keepdim=True)
    values = s["v_cache"][ids].permute(0, 2, 1, 4, 3).reshape(count, kv, pages * block, d)
    values = torch.where((j < new[:, None])[:, None, :, None], values, 0).float()
    outs = torch.matmul(scores, values) / torch.where(total > 0, total, 1.0)
    outs = outs.view(count, kv, most, h // kv, d).permute(0, 2, 1, 3, 4).reshape(count, most, h, d)
    return outs[at < new[:, None]].to(q.dtype)


def _plain_lora(s):
    t = torch.arange(s["x"].shape[0], dtype=torch.int32, device=s["x"].device)
    row = torch.searchsorted(s["cu"], t, right=True) - 1
    ids = s["adapters"][row]
    count, r, k = s["a"].shape
    # every row against every adapter, and the rows' own picked out: two plain products
    low = torch.matmul(s["x"].float(), s["a"].view(count * r, k).float().t()).view(-1, count, r)
    mine = ids[:, None] == torch.arange(count, device=ids.device)
    low = torch.where(mine[:, :, None], low * s["scaling"][:, None], 0.0)
    wide = s["b"].permute(0, 2, 1).reshape(count * r, -1).float()
    return torch.addmm(s["y"], low.view(-1, count * r), wide)


_plain = {"plan": _plain_plan, "store": _plain_store, "attention": _plain_attention, "lora": _plain_lora}


# -------------------------------------------------------------------------- the work
def work(case):
    ctx, new = _lengths(case)
    tokens, count = sum(new), case["requests"]
    if case["op"] == "plan":
        block = case["block"]
        have = [(c + block - 1) // block for c in ctx]
        fresh = sum((c + n + block - 1) // block - p for c, n, p in zip(ctx, new, have))
        old = sum(1 for c, n in zip(ctx, new) if n and c % block)
        words = _words(case) if case["tree"] else 0
        # lengths; table entries read, free pages read and written; offsets; slots, positions, parents and masks
        return {"bytes": 8 * count + 4 * old + 8 * fresh + 4 * (count + 1) + 8 * tokens
                + (4 + 8 * words) * tokens * bool(words), "flops": 2 * tokens}
    if case["op"] == "store":
        size = 2 if case["source"] == "same" else 4
        values = 2 * tokens * case["kv_heads"] * case["dim"]
        return {"bytes": values * (size + 2) + 4 * tokens, "flops": values}
    if case["op"] == "attention":
        h, kv, d = case["heads"], case["kv_heads"], case["dim"]
        cached = sum(c + n for c, n in zip(ctx, new)) * kv * d * 2 * 2
        return {"bytes": cached + 2 * tokens * h * d * 2 + sum((c + n) // case["block"] + 1 for c, n in zip(ctx, new)) * 4,
                "flops": sum(4 * n * (c + (n + 1) / 2) * h * d for c, n in zip(ctx, new))}
    n, k, r = case["n"], case["k"], case["rank"]
    ids = [-1 if b % 8 == 7 else b % case["adapters"] for b in range(count)]
    used = len({i for i in ids if i >= 0})
    share = sum(i >= 0 for i in ids) / count  # which requests go without an adapter is drawn
    return {"bytes": 2 * used * r * (n + k) + share * tokens * k * 2 + 8 * tokens * n,
            "flops": share * tokens * 2 * r * (n + k)}


# ------------------------------------------------- the definitions, in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return {"plan": _exact_plan, "store": _exact_store, "attention": _exact_attention,
            "lora": _exact_lora}[case["op"]](s)


def _exact_plan(s):
    ctx, new, free = (s[x].cpu().tolist() for x in ("ctx", "new", "free"))
    table, block, tokens = s["table"].cpu().numpy().astype(np.int64), s["case"]["block"], s["tokens"]
    parents = s["parents"].cpu().tolist() if s["parents"] is not None else None
    slots, positions = np.full(tokens, -1, np.int64), np.full(tokens, -1, np.int64)
    mask = np.zeros((tokens, max(1, s["words"])), np.uint64)
    cu, head, refused = [0], int(s["head"].item()), 0
    first, needed = head, 0
    for b, (c, n) in enumerate(zip(ctx, new)):
        start = cu[-1]
        cu.append(start + n)
        have, after = -(-c // block), -(-(c + n) // block)
        need = after - have if after <= table.shape[1] else 0
        needed += need
        ok = after <= table.shape[1] and cu[-1] <= tokens and (need == 0 or first + needed <= len(free))
        refused += not ok
        if ok:
            for p in range(need):
                table[b, have + p] = free[first + needed - need + p]
            head += need
        for i in range(n):
            depth = i
            if parents is not None:
                depth, up = 0, i
                while up >= 0:
                    mask[start + i, up // 64] |= np.uint64(1) << np.uint64(up % 64)
                    up = parents[start + up]
                    depth += up >= 0
            positions[start + i] = c + depth
            if ok:
                slots[start + i] = table[b, (c + i) // block] * block + (c + i) % block
    outs = {"table": table.astype(np.int32), "cu": np.array(cu, np.int32), "slots": slots.astype(np.int32),
            "positions": positions.astype(np.int32), "counts": np.array([cu[-1], head, refused], np.int32)}
    return outs | ({"mask": mask.view(np.int64)} if parents is not None else {})


def _exact_store(s):
    block = s["case"]["block"]
    outs = {"k_cache": s["k_cache"].double(), "v_cache": s["v_cache"].double()}
    slots = s["slots"].cpu().tolist()
    keep = [t for t, slot in enumerate(slots) if slot >= 0]
    rows = torch.tensor(keep, device="cuda")
    page = torch.tensor([slots[t] // block for t in keep], device="cuda")
    cell = torch.tensor([slots[t] % block for t in keep], device="cuda")
    outs["k_cache"].transpose(1, 2)[page, cell] = s["k"].double()[rows]
    outs["v_cache"].permute(0, 3, 1, 2)[page, cell] = s["v"].double()[rows]
    return outs


def _exact_attention(s):
    case, cu, ctx = s["case"], s["cu"].cpu().tolist(), s["ctx"].cpu().tolist()
    d, block, group = case["dim"], case["block"], case["heads"] // case["kv_heads"]
    outs = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    for b, c in enumerate(ctx):
        start, n = cu[b], cu[b + 1] - cu[b]
        if n == 0:
            continue
        ids = s["table"][b, :-(-(c + n) // block)].long()
        seen = torch.ones((n, c + n), dtype=torch.bool, device="cuda")
        if s["mask"] is None:
            seen[:, c:] = torch.ones((n, n), device="cuda").tril() > 0
        else:
            rows = s["mask"][start:start + n].cpu().numpy().view(np.uint8)
            bits = np.unpackbits(rows.reshape(n, -1), axis=1, bitorder="little")[:, :n]
            seen[:, c:] = torch.from_numpy(bits.astype(bool)).to("cuda")
        for h in range(case["kv_heads"]):
            keys = s["k_cache"][ids, h].reshape(-1, d)[:c + n].double()
            values = s["v_cache"][ids, h].transpose(1, 2).reshape(-1, d)[:c + n].double()
            for x in range(h * group, (h + 1) * group):
                z = s["q"][start:start + n, x].double() @ keys.t() / math.sqrt(d)
                z = torch.where(seen, z, -math.inf)
                outs[start:start + n, x] = torch.exp(z - torch.logsumexp(z, 1, keepdim=True)) @ values
    return outs


def _exact_lora(s):
    cu, ids = s["cu"].cpu().tolist(), s["adapters"].cpu().tolist()
    outs = s["y"].double()
    for b, i in enumerate(ids):
        if i >= 0:
            x = s["x"][cu[b]:cu[b + 1]].double()
            outs[cu[b]:cu[b + 1]] += s["scaling"][i].double() * ((x @ s["a"][i].double().t()) @ s["b"][i].double().t())
    return outs
