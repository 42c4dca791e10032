"""Plain forms of the serving operators in Python integers and 64-bit floats.

Written from the definitions, one request, token and key at a time: the page plan
of a step, the store into the paged cache, attention of drafted tokens over it and
low-rank adapters.  Arrays are NumPy; values of 16-bit types come as float64.
"""

import numpy as np


def page_plan(ctx, new, free, head, table, block, blocks, tokens, parents=None, words=0):
    """Returns (table, cu, slots, positions, mask or None, counts)."""
    table = np.array(table, np.int64, copy=True)
    width = table.shape[1]
    ctx = [max(int(c), 0) for c in ctx]
    new = [max(int(n), 0) for n in new]
    slots = np.full(tokens, -1, np.int64)
    positions = np.full(tokens, -1, np.int64)
    mask = np.zeros((tokens, words), np.uint64) if parents is not None else None
    starts, needed, taken, refused = [0], 0, 0, 0
    left = max(len(free) - max(head, 0), 0)
    for b, (c, n) in enumerate(zip(ctx, new)):
        start = starts[-1]
        starts.append(start + n)
        have, after = -(-c // block), -(-(c + n) // block)
        wide = after <= width
        need = after - have if wide else 0
        first = needed
        needed += need
        ok = wide and starts[-1] <= tokens and (need == 0 or needed <= left)
        if ok:
            for j in range(need):
                table[b, have + j] = free[head + first + j]
            if need:
                taken = needed
        else:
            refused += 1
        for i in range(n):
            row = start + i
            if row >= tokens:
                break
            depth, sound = i, True
            if parents is not None:
                chain, at = [], i
                sound = i < 64 * words
                while sound:
                    chain.append(at)
                    up = int(parents[start + at])
                    if up == -1:
                        break
                    sound = 0 <= up < at
                    at = up
                depth = len(chain) - 1
                if sound:
                    for j in chain:
                        mask[row, j // 64] |= np.uint64(1) << np.uint64(j % 64)
            if not sound:
                continue
            positions[row] = c + depth
            if ok:
                page = int(table[b, (c + i) // block])
                if 0 <= page < blocks:
                    slots[row] = page * block + (c + i) % block
    cu = np.minimum(np.array(starts, np.int64), tokens)
    counts = np.array([min(starts[-1], tokens + 1), max(head, 0) + taken, refused], np.int64)
    return table, cu, slots, positions, mask, counts


def ancestors(parents):
    """Boolean [n, n]: token i sees j if j is i or one of its ancestors."""
    n = len(parents)
    seen = np.zeros((n, n), bool)
    for i in range(n):
        j = i
        while j >= 0:
            seen[i, j] = True
            j = int(parents[j])
    return seen


def pack_mask(seen, words):
    """uint64 rows [n, words] of a boolean [n, n] (columns past 64 * words are lost)."""
    rows = np.zeros((len(seen), words), np.uint64)
    for i, j in zip(*np.nonzero(seen)):
        if j < 64 * words:
            rows[i, j // 64] |= np.uint64(1) << np.uint64(j % 64)
    return rows


def gather(k_cache, v_cache, pages, count):
    """Keys and values [count, heads, dim] of the first `count` positions of `pages`."""
    block = k_cache.shape[2]
    keys = [k_cache[pages[p // block], :, p % block] for p in range(count)]
    values = [v_cache[pages[p // block], :, :, p % block] for p in range(count)]
    shape = (0, k_cache.shape[1], k_cache.shape[3])
    return (np.stack(keys) if count else np.zeros(shape)), (np.stack(values) if count else np.zeros(shape))


def tree_attention(q, keys, values, ctx, seen, scale):
    """One request: q [n, heads, dim], keys and values [ctx + n, kv_heads, dim], seen
    boolean [n, n] over the new tokens.  Returns (out, weighted mean of |values|)."""
    n, heads, dim = q.shape
    group = heads // keys.shape[1]
    out, size = np.zeros(q.shape), np.zeros(q.shape)
    for i in range(n):
        visible = np.concatenate([np.ones(ctx, bool), seen[i]])
        if not visible.any():
            continue
        for h in range(heads):
            z = scale * (keys[visible, h // group] @ q[i, h])
            w = np.exp(z - z.max())
            v = values[visible, h // group]
            out[i, h] = w @ v / w.sum()
            size[i, h] = w @ np.abs(v) / w.sum()
    return out, size


def lora_add(y, x, a, b, scaling, ids, cu):
    """Returns (y with the adapters' share, the sums of the absolute products)."""
    out, size = np.array(y, np.float64, copy=True), np.zeros(np.shape(y))
    for r, i in enumerate(ids):
        if 0 <= i < len(a):
            rows = slice(int(cu[r]), int(cu[r + 1]))
            out[rows] += scaling[i] * ((x[rows] @ a[i].T) @ b[i].T)
            size[rows] += abs(scaling[i]) * ((np.abs(x[rows]) @ np.abs(a[i]).T) @ np.abs(b[i]).T)
    return out, size
