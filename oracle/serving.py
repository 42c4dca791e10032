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


def rope(x, positions, freqs, weight=None, eps=1e-6, interleaved=False):
    """Heads x [tokens, heads, dim], normed (with a weight) and turned by their positions."""
    x = np.array(x, np.float64, copy=True)
    pairs = len(freqs)
    for t in range(x.shape[0]):
        for h in range(x.shape[1]):
            if weight is not None:
                x[t, h] *= np.asarray(weight, np.float64) / np.sqrt(np.mean(x[t, h] ** 2) + eps)
            for i in range(pairs):
                a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + pairs)
                angle = float(positions[t]) * float(freqs[i])
                u, v = x[t, h, a], x[t, h, b]
                x[t, h, a] = u * np.cos(angle) - v * np.sin(angle)
                x[t, h, b] = v * np.cos(angle) + u * np.sin(angle)
    return x


def softmax(z):
    e = np.exp(z - z.max())
    return e / e.sum()


def verify(logits, draft, accept, sample, parents=None, probs=None, temperature=1.0):
    """One request: (path of accepted rows, next token).  logits [n, vocab]; row 0 is decided."""
    n = len(draft)
    if n == 0:
        return [], -1
    path, logits = [0], np.asarray(logits, np.float64)
    while True:
        end = path[-1]
        row = logits[end]
        if np.isnan(row).any() or not np.isfinite(row.max()):
            return path, -1
        children = [j for j in range(end + 1, n) if (parents[j] == end if parents is not None else j == end + 1)]
        if not temperature > 0:
            token = int(np.argmax(row))
            go = next((j for j in children if draft[j] == token), None)
            if go is None:
                return path, token
            path.append(go)
            continue
        z = np.full(len(row), -np.inf)  # (-inf excludes a token at an infinite temperature too)
        z[row > -np.inf] = row[row > -np.inf] / np.float64(temperature)
        p = softmax(z)
        q = None
        if probs is not None:
            q = np.where(probs[end] > 0, probs[end].astype(np.float64), 0.0)
        go = None
        for j in children:
            x = int(draft[j])
            if 0 <= x < len(row):
                if float(accept[j]) * (p.sum() if q is None else q[x]) < p[x]:
                    go = j
                    break
                if q is None:
                    p[x] = 0.0
            if q is not None:
                p = np.maximum(p - q, 0.0)
        if go is not None:
            path.append(go)
            continue
        total = np.cumsum(p)
        if total[-1] == 0.0:
            return path, int(np.argmax(row))
        at = int(np.searchsorted(total, float(sample) * total[-1], side="right"))
        return path, min(at, int(np.nonzero(p)[0][-1]))


def page_keep(path, kept, ctx, cu, slots, free, head, table, block, blocks):
    """Returns (moves as (from slot, to slot), lengths, free list, table, counts)."""
    table, free = np.array(table, np.int64, copy=True), np.array(free, np.int64, copy=True)
    valid = lambda s: 0 <= s < blocks * block
    moves, lens, gone = [], [], []
    for b in range(len(kept)):
        start, n, c = int(cu[b]), int(cu[b + 1] - cu[b]), max(int(ctx[b]), 0)
        refused = n == 0 or not valid(slots[start])
        k = 0
        while not refused and k < min(int(kept[b]), n):
            i = int(path[start + k]) if path is not None else k
            i = i if k < i < n else k  # (any other index leaves the place as it is)
            if not (valid(slots[start + i]) and valid(slots[start + k])):
                break  # never stored
            if i > k:
                moves.append((int(slots[start + i]), int(slots[start + k])))
            k += 1
        lens.append(c + k)
        if refused:
            continue
        for col in range(-(-(c + k) // block), min(-(-(c + n) // block), table.shape[1])):
            slot = int(slots[start + max(col * block, c) - c])
            page = slot // block if valid(slot) else int(table[b, col])  # (the plan wrote it there)
            if 0 <= page < blocks:
                gone.append(page)
                table[b, col] = -1
    free[head - len(gone):head] = gone
    return moves, np.array(lens), free, table, np.array([head - len(gone), len(gone)])


def page_fork(src, dst, lens, free, head, table, shares, block, blocks):
    """Returns (copies as (from page, to page, tokens), lengths, table, shares, counts)."""
    table, shares, old = np.array(table, np.int64, copy=True), np.array(shares, np.int64, copy=True), np.array(lens)
    lens, copies, refused, taken, named = old.copy(), [], 0, 0, set()
    for a, b in zip(src, dst):
        a, b = int(a), int(b)
        ok = 0 <= a < len(old) and 0 <= b < len(old) and b not in named
        if 0 <= b < len(old):
            named.add(b)
        ok = ok and old[a] > 0 and old[b] <= 0 and -(-int(old[a]) // block) <= table.shape[1]
        rest = int(old[a]) % block if ok else 0
        if ok and rest:
            taken += 1
            ok = head + taken <= len(free)
        if not ok:
            refused += 1
            continue
        full = int(old[a]) // block
        for c in range(full):
            table[b, c] = table[a, c]
            if 0 <= table[a, c] < blocks:
                shares[table[a, c]] += 1
        if rest:
            fresh = int(free[head + taken - 1])
            if 0 <= table[a, full] < blocks and 0 <= fresh < blocks:
                copies.append((int(table[a, full]), fresh, rest))
            table[b, full] = fresh
        lens[b] = old[a]
    return copies, lens, table, shares, np.array([min(head + taken, len(free)), refused])


def page_free(rows, lens, free, head, table, shares, block, blocks):
    """Returns (lengths, free list, table, shares, counts)."""
    table, shares, free, lens = (np.array(x, np.int64, copy=True) for x in (table, shares, free, lens))
    gone, seen = set(), set()
    for r in map(int, rows):
        if not 0 <= r < len(lens) or r in seen:
            continue
        seen.add(r)
        for c in range(min(-(-max(int(lens[r]), 0) // block), table.shape[1])):
            page = int(table[r, c])
            table[r, c] = -1
            if 0 <= page < blocks:
                shares[page] -= 1
                if shares[page] < 0:
                    gone.add(page)
        lens[r] = 0
    gone = sorted(gone)
    shares[gone] = 0
    free[head - len(gone):head] = gone
    return lens, free, table, shares, np.array([head - len(gone), len(gone)])
