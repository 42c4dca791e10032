"""Verifying drafted trees on compressed layers: the serving operators together.

Two attention layers whose projections stay compressed serve a batch of requests, each
with an adapter of its own (or none):

  1. a prompt step: pages for every request's prompt, rotated keys and values into them,
     attention of the whole prompts, the first token of each answer;
  2. verify steps: every request brings a tree of drafted tokens (of a draft that skips the
     layers); one pass through the layers gives each node its output, seeing what was kept
     and its own ancestors only;
  3. after each, the layers' logits say which drafts stand and what follows them.  Keys and
     values of the accepted nodes move to the places behind the cached tokens, and the pages
     that only the other nodes needed go back to the free list;
  4. at the end a request is forked: two answers share its full pages for a step, then the
     second one ends and gives back what no other holds.

A fused projection costs almost the same for one row as for 64 (each weight is decoded
once for all rows), which is why drafted tokens are worth verifying in trees.

``python examples/verify_step.py`` runs it on cuda:0 and checks the outputs of all steps
against a plain computation in float64 on the decompressed weights, and what was accepted
against the definition of it on the same logits.
"""

import os
import sys

import numpy as np
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import decode_gemm_tile_amd as dgt  # noqa: E402
from oracle import serving  # noqa: E402

HIDDEN, HEADS, KV_HEADS, DIM, LAYERS = 512, 8, 2, 64, 2
QKV = (HEADS + 2 * KV_HEADS) * DIM
BLOCK, BLOCKS, WIDTH = 16, 256, 32
RANK, ADAPTERS = 16, 3
VOCAB = 512


class Projection:
    """A compressed weight matrix and the adapters beside it."""

    def __init__(self, n, k, gen, gain=1.0):
        w = (torch.randn((n, k), generator=gen) * (gain * k ** -0.5)).to(torch.bfloat16)
        codes = w.view(torch.int16).numpy().view(np.uint16)
        self.layer = dgt.DeviceLayer(dgt.dgt_compress_layer(dgt.DGT_FMT_BF16_SPLIT, codes, 128, 64, 64))
        self.a = (torch.randn((ADAPTERS, RANK, k), generator=gen) * k ** -0.5).to(torch.bfloat16).cuda()
        self.b = (torch.randn((ADAPTERS, n, RANK), generator=gen) * 0.1).to(torch.bfloat16).cuda()
        self.scaling = torch.full((ADAPTERS,), 2.0, device="cuda")

    def __call__(self, x, adapters, cu):
        y = dgt.dgt_fused_decode_gemm(self.layer, x)
        return dgt.dgt_lora_add(y, x, self.a, self.b, self.scaling, adapters, cu)

    def plain(self, x, adapters, cu):
        """The same in float64, from the decompressed weights."""
        w = dgt.dgt_decode_tiles(self.layer).view(torch.bfloat16).double()
        y = x.double() @ w.t()
        for r, i in enumerate(adapters.tolist()):
            if 0 <= i < ADAPTERS:
                rows = slice(int(cu[r]), int(cu[r + 1]))
                y[rows] += self.scaling[i].double() * (x[rows].double() @ self.a[i].double().t()
                                                       @ self.b[i].double().t())
        return y


class Server:
    """The layers, their paged caches and the bookkeeping of the pages, all on the GPU."""

    def __init__(self, requests, seed=0, spare=0):
        """spare: rows of the table for requests that are forked later."""
        gen = torch.Generator().manual_seed(seed)
        self.qkv = [Projection(QKV, HIDDEN, gen) for _ in range(LAYERS)]
        self.out = [Projection(HIDDEN, HEADS * DIM, gen) for _ in range(LAYERS)]
        self.norms = [(1 + 0.1 * torch.randn((2, DIM), generator=gen)).cuda() for _ in range(LAYERS)]
        self.freqs = (10000.0 ** -(torch.arange(DIM // 2, dtype=torch.float64) / (DIM // 2))).cuda()
        self.embed = torch.randn((VOCAB, HIDDEN), generator=gen).to(torch.bfloat16).cuda()
        self.head_layer = Projection(VOCAB, HIDDEN, gen, gain=4.0)
        requests += spare
        # page numbers are shared by the layers, so one table serves all of them
        self.k = torch.zeros((LAYERS, BLOCKS, KV_HEADS, BLOCK, DIM), dtype=torch.bfloat16, device="cuda")
        self.v = torch.zeros((LAYERS, BLOCKS, KV_HEADS, DIM, BLOCK), dtype=torch.bfloat16, device="cuda")
        self.table = torch.full((requests, WIDTH), -1, dtype=torch.int32, device="cuda")
        self.free = torch.randperm(BLOCKS, generator=gen, dtype=torch.int32).cuda()
        self.head = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.shares = torch.zeros(BLOCKS, dtype=torch.int32, device="cuda")  # holders besides the first
        self.ws = dgt.alloc_workspace(dgt.dgt_page_free_workspace(BLOCKS)).zero_()
        self.lens = torch.zeros(requests, dtype=torch.int32, device="cuda")
        self.adapters = torch.tensor([i % (ADAPTERS + 1) - 1 for i in range(requests)], dtype=torch.int32,
                                     device="cuda")

    def step(self, x, new, parents=None):
        """One pass of the new rows x [tokens, HIDDEN] through the layers."""
        p = dgt.dgt_page_plan(self.lens, new, self.free, self.head, self.table, BLOCK, BLOCKS, x.shape[0],
                              parents=parents)
        self.head = p.counts[1:2]
        for i in range(LAYERS):
            qkv = self.qkv[i](x, self.adapters, p.cu).view(-1, HEADS + 2 * KV_HEADS, DIM)
            q = dgt.dgt_rope_store(qkv[:, :HEADS], qkv[:, HEADS:HEADS + KV_HEADS], qkv[:, HEADS + KV_HEADS:],
                                   p.positions, p.slots, self.freqs, self.k[i], self.v[i],
                                   q_weight=self.norms[i][0], k_weight=self.norms[i][1])
            if parents is None:
                a = dgt.dgt_chunk_attention(q, self.k[i], self.v[i], self.table, self.lens, p.cu)
            else:
                a = dgt.dgt_tree_attention(q, self.k[i], self.v[i], self.table, self.lens, p.cu, mask=p.mask)
            x = x + self.out[i](a.view(-1, HEADS * DIM), self.adapters, p.cu).to(torch.bfloat16)
        return x, p

    def logits(self, x):
        return dgt.dgt_fused_decode_gemm(self.head_layer.layer, x)

    def accept(self, p, path, kept):
        """Keep the first kept[b] rows of each request's path: their keys and values move behind the
        cached tokens in all layers, and the pages past them go back to the free list."""
        counts = dgt.dgt_page_keep(kept, self.lens, p.cu, p.slots, self.free, self.head, self.table, self.k, self.v,
                                   path=path)
        self.head = counts[0:1]

    def keep(self, p, path_rows, path_lens):
        """The same for rows of the whole step, path_lens of each request, in order."""
        path = torch.full_like(p.slots, -1)
        request = torch.repeat_interleave(torch.arange(len(path_lens), device="cuda"), path_lens)
        at = torch.arange(len(path_rows), device="cuda") - (path_lens.cumsum(0) - path_lens)[request]
        first = p.cu[request]
        path[first + at] = (path_rows - first).int()
        self.accept(p, path, path_lens)

    def fork(self, src, dst):
        """Rows `dst` of the table become requests that hold what rows `src` hold."""
        counts = dgt.dgt_page_fork(src, dst, self.lens, self.free, self.head, self.table, self.shares, self.k, self.v)
        self.head = counts[0:1]
        self.adapters[dst.long()] = self.adapters[src.long()]
        return counts

    def end(self, rows):
        counts = dgt.dgt_page_free(rows, self.lens, self.free, self.head, self.table, self.shares, BLOCK, ws=self.ws)
        self.head = counts[0:1]


def turned(x, weight, positions, freqs):
    """Heads x [tokens, heads, DIM] normed and turned by their positions, in float64."""
    x = x * weight.double() * (x.square().mean(-1, keepdim=True) + 1e-6).rsqrt()
    angle = (positions.double()[:, None] * freqs)[:, None]
    u, v = x.chunk(2, -1)
    return torch.cat([u * angle.cos() - v * angle.sin(), v * angle.cos() + u * angle.sin()], -1)


def plain_step(server, x, history, new, parents):
    """The same step for one request in float64 with the same roundings to bf16 between the
    operators.  history: per layer (k, v) [ctx, KV_HEADS, DIM] of the cached tokens."""
    n = x.shape[0]
    seen = torch.zeros((n, n), dtype=torch.bool)
    for i in range(n):
        j = i
        while j >= 0:
            seen[i, j] = True
            j = int(parents[j])
    made = []
    positions = (seen.sum(1) - 1 + history[0][0].shape[0]).to(x.device)
    for i in range(LAYERS):
        qkv = server.qkv[i].plain(x, new["adapter"], new["cu"]).view(n, -1, DIM)
        q, k = (turned(y, w, positions, server.freqs).to(torch.bfloat16).double()
                for y, w in zip((qkv[:, :HEADS], qkv[:, HEADS:HEADS + KV_HEADS]), server.norms[i]))
        v = qkv[:, HEADS + KV_HEADS:].to(torch.bfloat16).double()
        keys = torch.cat([history[i][0], k]).repeat_interleave(HEADS // KV_HEADS, 1)
        values = torch.cat([history[i][1], v]).repeat_interleave(HEADS // KV_HEADS, 1)
        made.append((torch.cat([history[i][0], k]), torch.cat([history[i][1], v])))
        z = torch.matmul(q.permute(1, 0, 2), keys.permute(1, 2, 0).contiguous()) * DIM ** -0.5
        mask = torch.cat([torch.ones((n, keys.shape[0] - n), dtype=torch.bool), seen], 1).to(z.device)
        w = torch.softmax(z.masked_fill(~mask, float("-inf")), -1)
        a = torch.matmul(w, values.permute(1, 0, 2).contiguous()).permute(1, 0, 2).reshape(n, -1).to(torch.bfloat16)
        x = x + server.out[i].plain(a, new["adapter"], new["cu"]).to(torch.bfloat16)
    return x, made


def draft_tree(root, count, likely, rng):
    """A tree of drafted tokens under `root`: parents and tokens.  likely [VOCAB, 2]: the two
    tokens that the draft finds most likely after each."""
    parents, tokens, children = [-1], [root], [0]
    while len(parents) < count:
        up = int(rng.choice([j for j in range(len(parents)) if children[j] < 2]))
        tokens.append(int(likely[tokens[up], children[up]]))
        children[up] += 1
        parents.append(up)
        children.append(0)
    return parents, tokens


def main(requests=6, seed=0, steps=3):
    rng = np.random.default_rng(seed)
    s = Server(requests, seed, spare=1)
    rows = requests + 1  # the last one is empty until a request is forked into it
    dev = lambda a, t=torch.int32: torch.tensor(np.asarray(a), dtype=t, device="cuda")
    uniform = lambda n: dev(rng.random(n), torch.float32)
    # the draft: the head on the embeddings themselves
    likely = s.logits(s.embed).topk(2).indices.cpu().numpy()
    temperature = dev([(0.0, 1.0, 0.5)[i % 3] for i in range(rows)], torch.float32)

    worst, drafted, kept = 0.0, 0, 0

    def check(got, want):
        nonlocal worst
        worst = max(worst, float((got.double() - want.double()).norm() / want.double().norm()))

    def check_pages():
        # every page is either in the table, once more than it is shared, or still free
        held, free = s.table[s.table >= 0].long(), s.free[int(s.head):].long()
        holders = torch.bincount(held, minlength=BLOCKS)
        assert torch.equal(holders + torch.bincount(free, minlength=BLOCKS), s.shares.long() + 1)
        assert torch.equal((s.table >= 0).sum(1), (s.lens.long() + BLOCK - 1) // BLOCK)

    def follow(logits, tokens, cu, parents=None):
        """What the layers' logits accept, checked against its definition on the same logits."""
        accept, sample = uniform(len(tokens)), uniform(len(cu) - 1)
        flat = None if parents is None else dev(sum(parents, []))
        got = dgt.dgt_verify(logits, dev(tokens), dev(cu), accept, sample, parents=flat, temperature=temperature)
        for r in range(len(cu) - 1):
            part = slice(cu[r], cu[r + 1])
            path, token = serving.verify(logits[part].cpu().numpy(), tokens[part], accept[part].tolist(),
                                         float(sample[r]), None if parents is None else parents[r],
                                         temperature=float(temperature[r]))
            assert int(got.accepted[r]) == len(path) and got.path[part].tolist()[:len(path)] == path
            assert int(got.next[r]) == token
        return got

    prompt = np.append(rng.integers(3, 60, requests), 0)
    tokens = rng.integers(0, VOCAB, prompt.sum())
    x = s.embed[dev(tokens, torch.int64)]
    y, p = s.step(x, dev(prompt))
    assert int(p.counts[2]) == 0
    s.lens += dev(prompt)
    check_pages()
    cu = np.concatenate([[0], np.cumsum(prompt)])
    last = [int(c) - 1 for c in cu[1:-1]]
    # each answer's first token: the row of one token is decided, so a token follows it
    one_each = list(range(requests + 1)) + [requests]
    roots = follow(s.logits(y[last]), tokens[last], one_each).next.tolist()[:requests]
    history = []  # of each request, per layer: keys and values of its cached tokens
    for r in range(requests):
        empty = [(torch.zeros((0, KV_HEADS, DIM), dtype=torch.float64, device="cuda"),) * 2] * LAYERS
        chain = list(range(-1, int(prompt[r]) - 1))
        one = {"adapter": s.adapters[r:r + 1], "cu": [0, int(prompt[r])]}
        want, made = plain_step(s, x[cu[r]:cu[r + 1]], empty, one, chain)
        check(y[cu[r]:cu[r + 1]], want)
        history.append(made)

    def verify_step(roots):
        """One step of all requests: trees under `roots`, what is accepted is kept.  Returns the
        tokens that follow."""
        nonlocal drafted, kept
        live = len(roots)
        nodes = np.append(rng.integers(1, 20, live), np.zeros(rows - live, int))
        trees = [draft_tree(root, n, likely, rng) for root, n in zip(roots, nodes)] + [([], [])] * (rows - live)
        parents, tokens = [t[0] for t in trees], np.array(sum((t[1] for t in trees), []), np.int64)
        before = s.lens.tolist()
        x = s.embed[dev(tokens, torch.int64)]
        y, p = s.step(x, dev(nodes), parents=dev(sum(parents, [])))
        assert int(p.counts[2]) == 0
        logits = s.logits(y)
        cu = np.concatenate([[0], np.cumsum(nodes)]).tolist()
        verified = follow(logits, tokens, cu, parents)
        s.accept(p, verified.path, verified.accepted)
        check_pages()
        for r in range(live):
            one = {"adapter": s.adapters[r:r + 1], "cu": [0, int(nodes[r])]}
            want, made = plain_step(s, x[cu[r]:cu[r + 1]], history[r], one, parents[r])
            check(y[cu[r]:cu[r + 1]], want)
            # what was kept lies behind the cached tokens, in order
            path = verified.path[cu[r]:cu[r] + int(verified.accepted[r])].tolist()
            assert int(s.lens[r]) == before[r] + len(path)
            places = list(range(before[r])) + [before[r] + j for j in path]
            history[r] = [(k[places], v[places]) for k, v in made]
            pos = torch.arange(len(places), device="cuda")
            page = s.table[r, pos // BLOCK].long()
            for i in range(LAYERS):
                check(s.k[i][page, :, pos % BLOCK], history[r][i][0])
                check(s.v[i][page, :, :, pos % BLOCK], history[r][i][1])
            kept += len(path)
        drafted += len(x)
        return verified.next.tolist()[:live]

    for _ in range(steps):
        roots = verify_step(roots)

    # a second answer to the first request, for a step; the pages before it are shared
    counts = s.fork(dev([0]), dev([requests]))
    assert int(counts[1]) == 0 and int(s.lens[requests]) == int(s.lens[0])
    check_pages()
    history.append(history[0])
    verify_step(roots + [int(likely[roots[0], 0])])
    s.end(dev([requests]))
    assert int(s.lens[requests]) == 0 and int(s.shares.sum()) == 0
    check_pages()
    print("verify steps: %d requests, %d prompt rows, %d drafted rows in %d steps, %d kept; "
          "largest relative difference %.1e" % (requests, prompt.sum(), drafted, steps + 1, kept, worst))
    # bf16 roundings that fall the other way between the operators: a few of 2^-8 each
    assert worst < 2e-2, worst
    return worst


if __name__ == "__main__":
    main()
