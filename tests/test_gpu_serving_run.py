"""The serving operators as a program runs them: a step captured once and replayed over many
steps, against the same steps run eagerly on a state of their own."""

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

REQUESTS, HEADS, KV_HEADS, DIM, BLOCK, BLOCKS, WIDTH, LAYERS, VOCAB, TOKENS = 5, 8, 2, 64, 16, 96, 12, 2, 700, 48


class State:
    """A server's state and a step's inputs, in buffers that stay."""

    def __init__(self, trees):
        import torch
        import decode_gemm_tile_amd as dgt
        i32 = lambda *shape: torch.zeros(shape, dtype=torch.int32, device="cuda")
        f32 = lambda *shape: torch.zeros(shape, dtype=torch.float32, device="cuda")
        self.k = torch.zeros((LAYERS, BLOCKS, KV_HEADS, BLOCK, DIM), dtype=torch.bfloat16, device="cuda")
        self.v = torch.zeros((LAYERS, BLOCKS, KV_HEADS, DIM, BLOCK), dtype=torch.bfloat16, device="cuda")
        self.table, self.free, self.head = i32(REQUESTS, WIDTH) - 1, i32(BLOCKS), i32(1)
        self.free += torch.arange(BLOCKS, dtype=torch.int32, device="cuda")
        self.lens, self.shares = i32(REQUESTS), i32(BLOCKS)
        self.new, self.parents = i32(REQUESTS), i32(TOKENS) if trees else None
        self.qkv = f32(TOKENS, HEADS + 2 * KV_HEADS, DIM)
        self.logits, self.draft = f32(TOKENS, VOCAB), i32(TOKENS)
        self.draw, self.sample = f32(TOKENS), f32(REQUESTS)
        self.ends, self.src, self.dst = i32(2) - 1, i32(1), i32(1)
        self.freqs = 1000.0 ** -(torch.arange(DIM // 2, dtype=torch.float64, device="cuda") / (DIM // 2))
        self.weight = torch.linspace(0.5, 1.5, DIM, device="cuda")
        self.out = [torch.zeros((TOKENS, HEADS, DIM), dtype=torch.bfloat16, device="cuda") for _ in range(LAYERS)]
        self.free_ws = dgt.alloc_workspace(dgt.dgt_page_free_workspace(BLOCKS)).zero_()

    def put(self, inputs):
        import torch
        for name, a in inputs.items():
            getattr(self, name).copy_(torch.as_tensor(a))

    def step(self):
        import decode_gemm_tile_amd as dgt
        # what ended before this step, and a request that is forked into an empty row
        head = dgt.dgt_page_free(self.ends, self.lens, self.free, self.head, self.table, self.shares, BLOCK,
                                 ws=self.free_ws)[0:1]
        forked = dgt.dgt_page_fork(self.src, self.dst, self.lens, self.free, head, self.table, self.shares, self.k,
                                   self.v)
        p = dgt.dgt_page_plan(self.lens, self.new, self.free, forked[0:1], self.table, BLOCK, BLOCKS, TOKENS,
                              parents=self.parents)
        k, v = self.qkv[:, HEADS:HEADS + KV_HEADS], self.qkv[:, HEADS + KV_HEADS:]
        for i in range(LAYERS):
            q = dgt.dgt_rope_store(self.qkv[:, :HEADS], k, v, p.positions, p.slots, self.freqs, self.k[i], self.v[i],
                                   k_weight=self.weight if i else None)
            if self.parents is None:
                dgt.dgt_chunk_attention(q, self.k[i], self.v[i], self.table, self.lens, p.cu, out=self.out[i])
            else:
                dgt.dgt_tree_attention(q, self.k[i], self.v[i], self.table, self.lens, p.cu, mask=p.mask,
                                       out=self.out[i])
        self.verified = dgt.dgt_verify(self.logits, self.draft, p.cu, self.draw, self.sample, parents=self.parents)
        kept = dgt.dgt_page_keep(self.verified.accepted, self.lens, p.cu, p.slots, self.free, p.counts[1:2],
                                 self.table, self.k, self.v, path=self.verified.path)
        self.head.copy_(kept[0:1])
        self.plan = p

    def seen(self):
        """What a program sees of the state: the free list in front of its head is used up."""
        n = int(self.plan.cu[-1])
        return ([self.k, self.v, self.table, self.head, self.lens, self.shares, self.free[int(self.head):],
                 self.plan.counts, self.plan.cu, self.verified.path[:n], self.verified.accepted, self.verified.next]
                + [o[:n] for o in self.out])


def _inputs(rng, lens, trees, step):
    """Inputs of a step: some requests end, one is forked into an empty row, all rows that hold
    tokens (and one that does not yet) get some."""
    new = rng.integers(1, 9, REQUESTS)
    new[rng.integers(0, REQUESTS)] = 0
    ends = np.full(2, -1)
    if step % 3 == 2:
        ends[0] = int(rng.integers(0, REQUESTS))
        new[ends[0]] = 0
    src, dst = int(np.argmax(lens)), -1
    empty = [r for r in range(REQUESTS) if (lens[r] == 0 or r == ends[0]) and r != src]
    if empty and src != ends[0]:
        dst = empty[0]
    total = int(new.sum())
    draft = np.where(rng.random(TOKENS) < 0.9, 3, 7)
    logits = rng.standard_normal((TOKENS, VOCAB)).astype(np.float32)
    logits[:, 3] += 9  # most drafts are likely ones
    d = {"new": new, "ends": ends, "src": [src], "dst": [dst], "draft": draft, "logits": logits,
         "qkv": rng.standard_normal((TOKENS, HEADS + 2 * KV_HEADS, DIM)).astype(np.float32),
         "draw": rng.random(TOKENS).astype(np.float32), "sample": rng.random(REQUESTS).astype(np.float32)}
    if trees:
        parents = [int(rng.integers(max(-1, i - 3), i)) if i else -1 for n in new for i in range(n)]
        d["parents"] = parents + [-1] * (TOKENS - total)
    return d


@pytest.mark.parametrize("trees", [False, True])
def test_captured_steps_are_the_eager_ones(trees):
    import torch
    rng = np.random.default_rng(11 + trees)
    eager, captured = State(trees), State(trees)
    first = _inputs(rng, np.zeros(REQUESTS, int), trees, 0)
    # (two runs of one step before the capture, as a program warms up; their state is put back)
    kept = {n: getattr(captured, n).clone() for n in ("k", "v", "table", "free", "head", "lens", "shares")}
    captured.put(first)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        captured.step()
        captured.step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured.step()
    captured.put(kept)
    accepted = forks = 0
    for step in range(12):
        inputs = first if step == 0 else _inputs(rng, eager.lens.cpu().numpy(), trees, step)
        eager.put(inputs)
        captured.put(inputs)
        before = eager.lens.clone()
        eager.step()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(eager.seen(), captured.seen()):
            assert torch.equal(a, b)
        assert int(eager.plan.counts[2]) == 0
        # every page is in the table, once more than it is shared, or free
        held, free = eager.table[eager.table >= 0].long(), eager.free[int(eager.head):].long()
        assert torch.equal(torch.bincount(held, minlength=BLOCKS) + torch.bincount(free, minlength=BLOCKS),
                           eager.shares.long() + 1)
        assert torch.equal((eager.table >= 0).sum(1), (eager.lens.long() + BLOCK - 1) // BLOCK)
        accepted += int(eager.verified.accepted.sum())
        forks += inputs["dst"][0] >= 0
    assert forks >= 2 and accepted > 12 * REQUESTS  # more than a row a request and step
