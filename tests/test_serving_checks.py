"""The serving operators refuse malformed arguments before anything is launched:
the binding by shape, dtype, layout and device (host tensors here, so every call
must raise), the C ABI by sizes, types and alignment."""

import pytest
import torch

import decode_gemm_tile_amd as dgt

I32, BF, F32 = torch.int32, torch.bfloat16, torch.float32


def _raises(match, fn, *a, **kw):
    with pytest.raises(ValueError, match=match):
        fn(*a, **kw)


def _plan_args(**over):
    a = dict(ctx_lens=torch.zeros(3, dtype=I32), new_lens=torch.zeros(3, dtype=I32),
             free_blocks=torch.zeros(5, dtype=I32), free_head=torch.zeros(1, dtype=I32),
             block_table=torch.zeros((3, 4), dtype=I32), block_size=16, num_blocks=20, tokens=6)
    return a | over


def test_page_plan_refusals():
    call = lambda **o: dgt.dgt_page_plan(**_plan_args(**o))
    _raises("arguments must be in GPU memory", call)
    _raises("new_lens has shape", call, new_lens=torch.zeros(2, dtype=I32))
    _raises("ctx_lens must be a 1-D", call, ctx_lens=torch.zeros((3, 1), dtype=I32))
    _raises("ctx_lens has dtype", call, ctx_lens=torch.zeros(3, dtype=torch.int64))
    _raises("free_head has shape", call, free_head=torch.zeros(2, dtype=I32))
    _raises("block_table has shape", call, block_table=torch.zeros((2, 4), dtype=I32))
    _raises("block_table must be contiguous", call, block_table=torch.zeros((4, 3), dtype=I32).t())
    _raises("parents has shape", call, parents=torch.zeros(5, dtype=I32))
    _raises("mask_words needs parents", call, mask_words=1)
    _raises("must not be negative", call, tokens=-1)
    out = dgt.PagePlan.empty(3, 6, 0, "cpu")
    _raises("arguments must be in GPU memory", call, out=out)
    _raises("out.slots has shape", call, tokens=7, out=out)
    _raises("out.mask is required", call, parents=torch.zeros(6, dtype=I32), out=out)


def _caches(blocks=4, heads=2, block=16, dim=64, dtype=BF):
    return torch.zeros((blocks, heads, block, dim), dtype=dtype), torch.zeros((blocks, heads, dim, block), dtype=dtype)


def test_kv_store_refusals():
    kc, vc = _caches()
    k, slots = torch.zeros((3, 2, 64)), torch.zeros(3, dtype=I32)
    call = dgt.dgt_kv_store
    _raises("arguments must be in GPU memory", call, k, k, slots, kc, vc)
    _raises("k has dtype", call, k.half(), k.half(), slots, kc, vc)
    _raises("v has dtype", call, k, k.to(BF), slots, kc, vc)
    _raises("v has shape", call, k, k[:2], slots, kc, vc)
    _raises("k has shape", call, torch.zeros((3, 3, 64)), k, slots, kc, vc)
    _raises("contiguous in its last", call, torch.zeros((3, 64, 2)).transpose(1, 2), k, slots, kc, vc)
    _raises("slots has dtype", call, k, k, slots.long(), kc, vc)
    _raises("v_cache has shape", call, k, k, slots, kc, kc)
    _raises("k_cache has dtype", call, k, k, slots, kc.float(), vc.float())
    _raises("k_cache must be contiguous", call, k, k, slots, kc[::2], vc[::2])


def _attn_args(**over):
    kc, vc = _caches()
    a = dict(q=torch.zeros((5, 4, 64), dtype=BF), k_cache=kc, v_cache=vc,
             block_table=torch.zeros((2, 3), dtype=I32), ctx_lens=torch.zeros(2, dtype=I32),
             cu=torch.zeros(3, dtype=I32))
    return a | over


def test_tree_attention_refusals():
    call = lambda **o: dgt.dgt_tree_attention(**_attn_args(**o))
    _raises("arguments must be in GPU memory", call)
    _raises("q has dtype", call, q=torch.zeros((5, 4, 64)))
    _raises("q has shape", call, q=torch.zeros((5, 4, 32), dtype=BF))
    _raises("not a multiple", call, q=torch.zeros((5, 3, 64), dtype=BF))
    _raises("q must be contiguous in its last", call, q=torch.zeros((5, 64, 4), dtype=BF).transpose(1, 2))
    _raises("cu has shape", call, cu=torch.zeros(2, dtype=I32))
    _raises("ctx_lens has shape", call, ctx_lens=torch.zeros(3, dtype=I32))
    _raises("mask has shape", call, mask=torch.zeros((4, 1), dtype=torch.int64))
    _raises("mask has dtype", call, mask=torch.zeros((5, 1), dtype=I32))
    _raises("at least one word", call, mask=torch.zeros((5, 0), dtype=torch.int64))
    _raises("out has dtype", call, out=torch.zeros((5, 4, 64)))
    _raises("ws has dtype", call, ws=torch.zeros(64))
    for shape, kv in (((5, 4, 260), 2), ((5, 4, 12), 2), ((5, 3, 64), 2)):
        with pytest.raises(dgt.DgtError):
            dgt.dgt_tree_attention_workspace(shape, kv, 2)


def _lora_args(**over):
    a = dict(y=torch.zeros((5, 40)), x=torch.zeros((5, 64), dtype=BF), a=torch.zeros((2, 16, 64), dtype=BF),
             b=torch.zeros((2, 40, 16), dtype=BF), scaling=torch.zeros(2), adapters=torch.zeros(3, dtype=I32),
             cu=torch.zeros(4, dtype=I32))
    return a | over


def test_lora_refusals():
    call = lambda **o: dgt.dgt_lora_add(**_lora_args(**o))
    _raises("arguments must be in GPU memory", call)
    _raises("y has dtype", call, y=torch.zeros((5, 40), dtype=BF))
    _raises("x has shape", call, x=torch.zeros((4, 64), dtype=BF))
    _raises("x has dtype", call, x=torch.zeros((5, 64)))
    _raises("a has shape", call, a=torch.zeros((2, 16, 32), dtype=BF))
    _raises("b has shape", call, b=torch.zeros((2, 16, 40), dtype=BF))
    _raises("scaling has shape", call, scaling=torch.zeros(3))
    _raises("cu has shape", call, cu=torch.zeros(3, dtype=I32))
    _raises("out has shape", call, out=torch.zeros((5, 41)))
    for t, r, n, k, rank in ((5, 3, 40, 64, 12), (5, 3, 40, 64, 264), (5, 3, 40, 60, 16), (5, 3, 0, 64, 16)):
        with pytest.raises(dgt.DgtError):
            dgt.dgt_lora_workspace(t, r, n, k, rank)


def test_c_abi_refusals():
    """Codes of the entry points themselves; nothing here gets as far as a launch."""
    L, p = dgt.lib(), 256  # an address that is aligned and never read
    plan = lambda ctx=p, requests=2, head=p, width=4, block=16, blocks=8, tokens=3, parents=None, words=0, \
        mask=None: L.dgt_page_plan(ctx, p, requests, p, 5, head, p, width, block, blocks, tokens, parents,
                                   words, p, p, p, mask, p, None)
    assert plan(ctx=None) == -1 and plan(head=None) == -1
    assert plan(block=24) == -2 and plan(block=4) == -2 and plan(block=2048) == -2
    assert plan(blocks=1 << 28) == -2 and plan(requests=8193) == -2 and plan(tokens=(1 << 28) + 1) == -2
    assert plan(width=1 << 28) == -2
    assert plan(parents=p) == -1 and plan(words=1) == -1 and plan(parents=p, words=1) == -1
    store = lambda k=p, source=3, heads=2, dim=64, cache=1, kc=p, blocks=8, block=16: L.dgt_kv_store(
        k, p, source, 128, 64, 128, 64, p, 3, heads, dim, cache, kc, p, blocks, block, None)
    assert store(k=None) == -1 and store(kc=260) == -1
    assert store(cache=3) == -8 and store(source=2) == -8 and store(source=0) == -8
    assert store(dim=60) == -2 and store(heads=0) == -2 and store(block=12) == -2 and store(dim=1032) == -2
    attn = lambda ty=1, q=p, qrow=256, block=16, heads=4, kv=2, dim=64, mask=None, words=0, scale=0.1, orow=256, \
        ws=p, size=1 << 30, blocks=8: L.dgt_tree_attention(
            ty, q, qrow, 64, p, p, blocks, block, p, 4, p, p, 2, 5, heads, kv, dim, mask, words, scale, p, orow,
            64, ws, size, None)
    assert attn(ty=3) == -8
    assert attn(q=None) == -1 and attn(q=264) == -1 and attn(ws=None) == -1 and attn(qrow=252) == -1
    assert attn(scale=0.0) == -1 and attn(scale=-1.0) == -1 and attn(scale=float("nan")) == -1
    assert attn(scale=float("inf")) == -1 and attn(orow=255) == -1
    assert attn(mask=p) == -1 and attn(words=1) == -1
    assert attn(block=20) == -2 and attn(dim=264) == -2 and attn(dim=20) == -2 and attn(heads=3) == -2
    assert attn(kv=0) == -2 and attn(blocks=0) == -2
    assert attn(size=dgt.dgt_tree_attention_workspace((5, 4, 64), 2, 2) - 1) == -4
    lora = lambda y=p, x=p, xrow=64, yrow=40, n=40, k=64, rank=16, out=512, orow=40, ws=p, size=1 << 30, \
        ids=p: L.dgt_lora_add(y, yrow, x, xrow, p, p, p, 2, ids, p, 3, 5, n, k, rank, out, orow, ws, size, None)
    assert lora(y=None) == -1 and lora(ids=None) == -1 and lora(x=264) == -1 and lora(ws=128) == -1
    assert lora(out=p, orow=48) == -1
    assert lora(rank=20) == -2 and lora(rank=264) == -2 and lora(k=60) == -2 and lora(n=0) == -2
    assert lora(xrow=56) == -2 and lora(xrow=68) == -2 and lora(yrow=39) == -2 and lora(orow=39) == -2
    assert lora(size=dgt.dgt_lora_workspace(5, 3, 40, 64, 16) - 1) == -4


def test_header_and_binding_agree_on_the_cleared_bytes():
    import os
    import re
    header = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "dgt.h")
    value = re.search(r"#define DGT_TREE_ATTENTION_ZEROED (\d+)", open(header).read()).group(1)
    assert int(value) == dgt.DGT_TREE_ATTENTION_ZEROED


def test_empty_calls_do_nothing():
    """No token: success without a launch (the pointers are never read)."""
    L = dgt.lib()
    assert L.dgt_kv_store(None, None, 3, 0, 0, 0, 0, None, 0, 2, 64, 1, None, None, 8, 16, None) == 0
    assert L.dgt_tree_attention(1, None, 0, 0, None, None, 8, 16, None, 4, None, None, 2, 0, 4, 2, 64, None, 0,
                                0.1, None, 0, 0, None, 0, None) == 0
    assert L.dgt_lora_add(None, 40, None, 64, None, None, None, 2, None, None, 3, 0, 40, 64, 16, None, 40, None,
                          0, None) == 0
