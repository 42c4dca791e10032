"""Verifying drafted trees on compressed layers: the serving operators together.

Two attention layers whose projections stay compressed serve a batch of requests, each
with an adapter of its own (or none):

  1. a prompt step: pages for every request's prompt, keys and values into them;
  2. verify steps: every request brings a tree of drafted tokens; one pass through the
     layers gives each node its output, seeing what was kept and its own ancestors only;
  3. after each, the nodes on one path of each tree are kept: their keys and values move
     to the places behind the cached tokens, and the pages that only the other nodes
     needed go back to the free list.

A fused projection costs almost the same for one row as for 64 (each weight is decoded
once for all rows), which is why drafted tokens are worth verifying in trees.

``python examples/verify_step.py`` runs it on cuda:0 and checks the outputs of all steps
against a plain computation in float64 on the decompressed weights.
"""

import os
import sys

import numpy as np
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import decode_gemm_tile_amd as dgt  # noqa: E402

HIDDEN, HEADS, KV_HEADS, DIM, LAYERS = 512, 8, 2, 64, 2
QKV = (HEADS + 2 * KV_HEADS) * DIM
BLOCK, BLOCKS, WIDTH = 16, 256, 32
RANK, ADAPTERS = 16, 3


class Projection:
    """A compressed weight matrix and the adapters beside it."""

    def __init__(self, n, k, gen):
        w = (torch.randn((n, k), generator=gen) * k ** -0.5).to(torch.bfloat16)
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

    def __init__(self, requests, seed=0):
        gen = torch.Generator().manual_seed(seed)
        self.qkv = [Projection(QKV, HIDDEN, gen) for _ in range(LAYERS)]
        self.out = [Projection(HIDDEN, HEADS * DIM, gen) for _ in range(LAYERS)]
        # one pool a layer; page numbers are shared, so one table serves all layers
        self.k = [torch.zeros((BLOCKS, KV_HEADS, BLOCK, DIM), dtype=torch.bfloat16, device="cuda")
                  for _ in range(LAYERS)]
        self.v = [torch.zeros((BLOCKS, KV_HEADS, DIM, BLOCK), dtype=torch.bfloat16, device="cuda")
                  for _ in range(LAYERS)]
        self.table = torch.full((requests, WIDTH), -1, dtype=torch.int32, device="cuda")
        self.free = torch.randperm(BLOCKS, generator=gen, dtype=torch.int32).cuda()
        self.head = torch.zeros(1, dtype=torch.int32, device="cuda")
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
            dgt.dgt_kv_store(qkv[:, HEADS:HEADS + KV_HEADS], qkv[:, HEADS + KV_HEADS:], p.slots, self.k[i], self.v[i])
            q = qkv[:, :HEADS].to(torch.bfloat16)
            a = dgt.dgt_tree_attention(q, self.k[i], self.v[i], self.table, self.lens, p.cu, mask=p.mask)
            x = x + self.out[i](a.view(-1, HEADS * DIM), self.adapters, p.cu).to(torch.bfloat16)
        return x, p

    def keep(self, p, path_rows, path_lens):
        """Keep the rows `path_rows` of the last step (path_lens of each request, in order):
        their keys and values move to the places right behind the cached tokens.  Pages past
        the kept tokens go back to the free list, in front of its head: the next plan counts a
        request's pages by its length and takes fresh ones from there on."""
        # the destinations are the slots of the first rows of each request
        at = torch.cat([p.cu[r] + torch.arange(n, device="cuda") for r, n in enumerate(path_lens.tolist())])
        src, dst = p.slots[path_rows].long(), p.slots[at]
        for k, v in zip(self.k, self.v):
            dgt.dgt_kv_store(k[src // BLOCK, :, src % BLOCK], v[src // BLOCK, :, :, src % BLOCK], dst, k, v)
        self.lens += path_lens
        pages = (self.lens + BLOCK - 1) // BLOCK
        surplus = (torch.arange(WIDTH, device="cuda") >= pages[:, None]) & (self.table >= 0)
        ids = self.table[surplus]
        self.head = self.head - len(ids)
        self.free[self.head + torch.arange(len(ids), device="cuda")] = ids
        self.table[surplus] = -1


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
    for i in range(LAYERS):
        qkv = server.qkv[i].plain(x, new["adapter"], new["cu"]).view(n, -1, DIM).to(torch.bfloat16).double()
        q, k, v = qkv[:, :HEADS], qkv[:, HEADS:HEADS + KV_HEADS], qkv[:, HEADS + KV_HEADS:]
        keys = torch.cat([history[i][0], k]).repeat_interleave(HEADS // KV_HEADS, 1)
        values = torch.cat([history[i][1], v]).repeat_interleave(HEADS // KV_HEADS, 1)
        made.append((torch.cat([history[i][0], k]), torch.cat([history[i][1], v])))
        z = torch.matmul(q.permute(1, 0, 2), keys.permute(1, 2, 0).contiguous()) * DIM ** -0.5
        mask = torch.cat([torch.ones((n, keys.shape[0] - n), dtype=torch.bool), seen], 1).to(z.device)
        w = torch.softmax(z.masked_fill(~mask, float("-inf")), -1)
        a = torch.matmul(w, values.permute(1, 0, 2).contiguous()).permute(1, 0, 2).reshape(n, -1).to(torch.bfloat16)
        x = x + server.out[i].plain(a, new["adapter"], new["cu"]).to(torch.bfloat16)
    return x, made


def main(requests=6, seed=0, steps=3):
    gen = torch.Generator().manual_seed(seed + 1)
    rng = np.random.default_rng(seed)
    s = Server(requests, seed)
    dev = lambda a: torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")

    def rows(count):
        return torch.randn((count, HIDDEN), generator=gen).to(torch.bfloat16).cuda()

    worst, drafted, kept = 0.0, 0, 0

    def check(got, want):
        nonlocal worst
        worst = max(worst, float((got.double() - want.double()).norm() / want.double().norm()))

    def check_pages():
        # every page is either in one request's table or still free
        held = s.table[s.table >= 0]
        free = s.free[int(s.head):]
        assert torch.equal(torch.cat([held, free]).sort().values, torch.arange(BLOCKS, dtype=torch.int32, device="cuda"))
        assert torch.equal((s.table >= 0).sum(1), (s.lens.long() + BLOCK - 1) // BLOCK)

    prompt = rng.integers(3, 60, requests)
    x = rows(int(prompt.sum()))
    y, p = s.step(x, dev(prompt))
    assert int(p.counts[2]) == 0
    s.lens += dev(prompt)
    check_pages()
    cu = np.concatenate([[0], np.cumsum(prompt)])
    history = []  # of each request, per layer: keys and values of its cached tokens
    for r in range(requests):
        empty = [(torch.zeros((0, KV_HEADS, DIM), dtype=torch.float64, device="cuda"),) * 2] * LAYERS
        chain = list(range(-1, int(prompt[r]) - 1))
        one = {"adapter": s.adapters[r:r + 1], "cu": [0, int(prompt[r])]}
        want, made = plain_step(s, x[cu[r]:cu[r + 1]], empty, one, chain)
        check(y[cu[r]:cu[r + 1]], want)
        history.append(made)

    for _ in range(steps):
        nodes = rng.integers(1, 20, requests)
        parents = [[-1] + [int(rng.integers(-1, i)) for i in range(1, n)] for n in nodes]
        before = s.lens.tolist()
        x = rows(int(nodes.sum()))
        y, p = s.step(x, dev(nodes), parents=dev(sum(parents, [])))
        assert int(p.counts[2]) == 0

        # each tree keeps the way to its last node
        paths = []
        for up in parents:
            way, j = [], len(up) - 1
            while j >= 0:
                way.append(j)
                j = up[j]
            paths.append(way[::-1])
        cu = np.concatenate([[0], np.cumsum(nodes)])
        s.keep(p, torch.tensor([cu[r] + j for r, w in enumerate(paths) for j in w], device="cuda"),
               dev([len(w) for w in paths]))
        check_pages()
        drafted, kept = drafted + len(x), kept + sum(map(len, paths))

        for r in range(requests):
            one = {"adapter": s.adapters[r:r + 1], "cu": [0, int(nodes[r])]}
            want, made = plain_step(s, x[cu[r]:cu[r + 1]], history[r], one, parents[r])
            check(y[cu[r]:cu[r + 1]], want)
            # what was kept lies behind the cached tokens, in order
            places = list(range(before[r])) + [before[r] + j for j in paths[r]]
            history[r] = [(k[places], v[places]) for k, v in made]
            pos = torch.arange(before[r], before[r] + len(paths[r]), device="cuda")
            page = s.table[r, pos // BLOCK].long()
            for i in range(LAYERS):
                check(s.k[i][page, :, pos % BLOCK], history[r][i][0][before[r]:])
                check(s.v[i][page, :, :, pos % BLOCK], history[r][i][1][before[r]:])
    print("verify steps: %d requests, %d prompt rows, %d drafted rows in %d steps, %d kept; "
          "largest relative difference %.1e" % (requests, prompt.sum(), drafted, steps, kept, worst))
    # bf16 roundings that fall the other way between the operators: a few of 2^-8 each
    assert worst < 2e-2, worst
    return worst


if __name__ == "__main__":
    main()
