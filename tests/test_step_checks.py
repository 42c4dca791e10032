"""Rotation, verification, page moves and chunk attention refuse malformed arguments before anything is
launched: the binding by shape, dtype, layout and device (host tensors here, so every call must raise),
the C ABI by sizes, types and alignment."""

import pytest
import torch

import decode_gemm_tile_amd as dgt

I32, BF, F32, F64 = torch.int32, torch.bfloat16, torch.float32, torch.float64


def _raises(match, fn, *a, **kw):
    with pytest.raises(ValueError, match=match):
        fn(*a, **kw)


def _caches(blocks=4, heads=2, block=16, dim=64, dtype=BF, front=()):
    return (torch.zeros(front + (blocks, heads, block, dim), dtype=dtype),
            torch.zeros(front + (blocks, heads, dim, block), dtype=dtype))


def _ints(*n):
    return torch.zeros(n, dtype=I32)


def test_rope_refusals():
    kc, vc = _caches()
    base = dict(q=torch.zeros((3, 4, 64)), k=torch.zeros((3, 2, 64)), v=torch.zeros((3, 2, 64)), positions=_ints(3),
                slots=_ints(3), freqs=torch.zeros(32, dtype=F64), k_cache=kc, v_cache=vc)
    call = lambda **o: dgt.dgt_rope_store(**(base | o))
    _raises("arguments must be in GPU memory", call)
    _raises("arguments must be in GPU memory", call, freqs=None, q_weight=torch.zeros(64))
    _raises("q has dtype", call, q=torch.zeros((3, 4, 64), dtype=torch.float16))
    _raises("q has shape", call, q=torch.zeros((3, 4, 32)))
    _raises("q must be a 3-D", call, q=torch.zeros((3, 256)))
    _raises("k has dtype", call, k=torch.zeros((3, 2, 64), dtype=BF))
    _raises("k has shape", call, k=torch.zeros((3, 3, 64)))
    _raises("v has shape", call, v=torch.zeros((2, 2, 64)))
    _raises("v must be contiguous in its last", call, v=torch.zeros((3, 64, 2)).transpose(1, 2))
    _raises("positions has dtype", call, positions=torch.zeros(3, dtype=torch.int64))
    _raises("slots has shape", call, slots=_ints(4))
    _raises("freqs has dtype", call, freqs=torch.zeros(32))
    _raises("freqs holds 33 pairs", call, freqs=torch.zeros(33, dtype=F64))
    _raises("q_weight has shape", call, q_weight=torch.zeros(32))
    _raises("k_weight has dtype", call, k_weight=torch.zeros(64, dtype=BF))
    _raises("q_out has dtype", call, q_out=torch.zeros((3, 4, 64)))
    _raises("v_cache has shape", call, v_cache=kc)


def test_chunk_attention_refusals():
    kc, vc = _caches()
    base = dict(q=torch.zeros((5, 4, 64), dtype=BF), k_cache=kc, v_cache=vc, block_table=_ints(2, 3), ctx_lens=_ints(2),
                cu=_ints(3))
    call = lambda **o: dgt.dgt_chunk_attention(**(base | o))
    _raises("arguments must be in GPU memory", call)
    _raises("q has dtype", call, q=torch.zeros((5, 4, 64)))
    _raises("not a multiple", call, q=torch.zeros((5, 3, 64), dtype=BF))
    _raises("cu has shape", call, cu=_ints(2))
    _raises("ctx_lens has dtype", call, ctx_lens=torch.zeros(2))
    _raises("block_table must be contiguous", call, block_table=_ints(3, 2).t())
    _raises("out has shape", call, out=torch.zeros((5, 4, 32), dtype=BF))
    _raises("ws has dtype", call, ws=torch.zeros(64))
    for shape, kv in (((5, 4, 260), 2), ((5, 4, 12), 2), ((5, 3, 64), 2)):
        with pytest.raises(dgt.DgtError):
            dgt.dgt_chunk_attention_workspace(shape, kv, 2)


def test_verify_refusals():
    base = dict(logits=torch.zeros((6, 50)), draft=_ints(6), cu=_ints(3), accept=torch.zeros(6), sample=torch.zeros(2))
    call = lambda **o: dgt.dgt_verify(**(base | o))
    _raises("arguments must be in GPU memory", call)
    _raises("arguments must be in GPU memory", call, parents=_ints(6), temperature=torch.zeros(2))
    _raises("logits must be a 2-D", call, logits=torch.zeros(50))
    _raises("logits has dtype", call, logits=torch.zeros((6, 50), dtype=F64))
    _raises("contiguous in its last", call, logits=torch.zeros((50, 6)).t())
    _raises("draft has dtype", call, draft=torch.zeros(6, dtype=torch.int64))
    _raises("draft has shape", call, draft=_ints(5))
    _raises("cu has shape", call, cu=_ints(2))
    _raises("accept has dtype", call, accept=torch.zeros(6, dtype=F64))
    _raises("sample must be a 1-D", call, sample=torch.zeros(()))
    _raises("parents has shape", call, parents=_ints(5))
    _raises("only taken for chains", call, parents=_ints(6), draft_probs=torch.zeros((6, 50)))
    _raises("draft_probs has dtype", call, draft_probs=torch.zeros((6, 50), dtype=BF))
    _raises("draft_probs has shape", call, draft_probs=torch.zeros((6, 49)))
    _raises("temperature has shape", call, temperature=torch.zeros(3))
    _raises("out.path has shape", call, out=dgt.Verified.empty(2, 5, "cpu"))
    _raises("ws has dtype", call, ws=torch.zeros(4))
    for tokens, vocab, requests in ((5, 0, 2), (5, (1 << 22) + 1, 2), (5, 10, 8193), ((1 << 20) + 1, 10, 2)):
        with pytest.raises(dgt.DgtError):
            dgt.dgt_verify_workspace(tokens, vocab, requests)


def test_page_moves_refusals():
    kc, vc = _caches(front=(3,))
    base = dict(kept=_ints(2), ctx_lens=_ints(2), cu=_ints(3), slots=_ints(5), free_blocks=_ints(9), free_head=_ints(1),
                block_table=_ints(2, 4), k_cache=kc, v_cache=vc)
    keep = lambda **o: dgt.dgt_page_keep(**(base | o))
    _raises("arguments must be in GPU memory", keep)
    _raises("arguments must be in GPU memory", keep, k_cache=kc[0], v_cache=vc[0], path=_ints(5))
    _raises("k_cache must be a 4-D or 5-D", keep, k_cache=kc[0, 0])
    _raises("k_cache has dtype", keep, k_cache=kc.float(), v_cache=vc.float())
    _raises("v_cache has shape", keep, v_cache=vc[:2])
    _raises("k_cache must be contiguous", keep, k_cache=kc[:, ::2], v_cache=vc[:, ::2])
    _raises("ctx_lens has shape", keep, ctx_lens=_ints(3))
    _raises("cu has shape", keep, cu=_ints(2))
    _raises("path has shape", keep, path=_ints(4))
    _raises("lens has dtype", keep, lens=torch.zeros(2))
    _raises("counts has shape", keep, counts=_ints(3))
    _raises("free_head has shape", keep, free_head=_ints(2))
    base2 = dict(src=_ints(2), dst=_ints(2), lens=_ints(3), free_blocks=_ints(9), free_head=_ints(1),
                 block_table=_ints(3, 4), shares=_ints(4), k_cache=kc, v_cache=vc)
    fork = lambda **o: dgt.dgt_page_fork(**(base2 | o))
    _raises("arguments must be in GPU memory", fork)
    _raises("dst has shape", fork, dst=_ints(3))
    _raises("src must be a 1-D", fork, src=_ints(2, 1))
    _raises("lens has shape", fork, lens=_ints(2))
    _raises("shares has shape", fork, shares=_ints(5))
    _raises("shares has dtype", fork, shares=torch.zeros(4))
    base3 = dict(rows=_ints(2), lens=_ints(3), free_blocks=_ints(9), free_head=_ints(1), block_table=_ints(3, 4),
                 shares=_ints(4), block_size=16)
    free = lambda **o: dgt.dgt_page_free(**(base3 | o))
    _raises("arguments must be in GPU memory", free)
    _raises("rows has dtype", free, rows=torch.zeros(2, dtype=torch.int64))
    _raises("lens has shape", free, lens=_ints(2))
    _raises("ws has dtype", free, ws=_ints(4))
    _raises("block_table must be a 2-D", free, block_table=_ints(4))


def test_c_abi_refusals():
    """Codes of the entry points themselves; nothing here gets as far as a launch."""
    L, p = dgt.lib(), 256  # an address that is aligned and never read
    rope = lambda q=p, source=3, tokens=3, heads=4, kv=2, dim=64, freqs=p, pairs=32, eps=1e-6, ty=1, out=p, orow=256, \
        kc=p, blocks=8, block=16: L.dgt_rope_store(q, p, p, source, 512, 64, 512, 64, 512, 64, p, p, tokens, heads, kv, dim,
                                                   freqs, pairs, 0, None, None, eps, ty, out, orow, 64, kc, p, blocks,
                                                   block, None)
    assert rope(q=None) == -1 and rope(freqs=None) == -1 and rope(out=264) == -1 and rope(kc=264) == -1
    assert rope(eps=-1.0) == -1 and rope(eps=float("nan")) == -1 and rope(orow=252) == -1
    assert rope(dim=60) == -2 and rope(dim=264) == -2 and rope(pairs=33) == -2 and rope(block=12) == -2
    assert rope(heads=0) == -2 and rope(kv=0) == -2 and rope(blocks=1 << 28) == -2 and rope(tokens=(1 << 20) + 1) == -2
    assert rope(ty=3) == -8 and rope(source=2) == -8 and rope(source=0) == -8
    chunk = lambda ty=1, q=p, qrow=256, block=16, heads=4, kv=2, dim=64, scale=0.1, orow=256, ws=p, size=1 << 40, blocks=8, \
        table=p: L.dgt_chunk_attention(ty, q, qrow, 64, p, p, blocks, block, table, 4, p, p, 2, 5, heads, kv, dim, scale, p,
                                       orow, 64, ws, size, None)
    assert chunk(ty=3) == -8 and chunk(q=None) == -1 and chunk(q=264) == -1 and chunk(ws=None) == -1 and chunk(ws=272) == -1
    assert chunk(table=None) == -1 and chunk(qrow=252) == -1 and chunk(orow=255) == -1
    assert chunk(scale=0.0) == -1 and chunk(scale=float("inf")) == -1 and chunk(scale=float("nan")) == -1
    assert chunk(block=20) == -2 and chunk(dim=264) == -2 and chunk(dim=20) == -2 and chunk(heads=3) == -2
    assert chunk(kv=0) == -2 and chunk(blocks=0) == -2
    assert chunk(size=dgt.dgt_chunk_attention_workspace((5, 4, 64), 2, 2) - 1) == -4
    verify = lambda ty=3, logits=p, row=50, probs=None, prow=50, parents=None, cu=p, requests=2, tokens=5, vocab=50, ws=p, \
        size=1 << 40: L.dgt_verify(ty, logits, row, p, probs, prow, parents, cu, None, p, p, requests, tokens, vocab, p, p,
                                   p, ws, size, None)
    assert verify(ty=0) == -8 and verify(probs=p, parents=p) == -8
    assert verify(logits=None) == -1 and verify(cu=None) == -1 and verify(ws=None) == -1 and verify(ws=264) == -1
    assert verify(vocab=0) == -2 and verify(row=49) == -2 and verify(probs=p, prow=49) == -2 and verify(requests=8193) == -2
    assert verify(size=dgt.dgt_verify_workspace(5, 50, 2) - 1) == -4
    keep = lambda kept=p, slots=p, requests=2, tokens=5, free=p, head=p, table=p, layers=1, heads=2, dim=64, blocks=8, \
        block=16, kc=p, counts=p, width=4: L.dgt_page_keep(None, kept, p, p, slots, requests, tokens, free, 9, head, table,
                                                           width, layers, heads, dim, blocks, block, kc, p, p, counts, None)
    assert keep(kept=None) == -1 and keep(slots=None) == -1 and keep(free=None) == -1 and keep(head=None) == -1
    assert keep(table=None) == -1 and keep(kc=None) == -1 and keep(kc=264) == -1 and keep(counts=None) == -1
    assert keep(layers=0) == -2 and keep(heads=0) == -2 and keep(dim=12) == -2 and keep(dim=1032) == -2
    assert keep(block=4) == -2 and keep(requests=8193) == -2 and keep(width=1 << 28) == -2 and keep(blocks=1 << 28) == -2
    fork = lambda src=p, forks=2, lens=p, requests=3, width=4, shares=p, layers=1, block=16, blocks=8, head=p: \
        L.dgt_page_fork(src, p, forks, lens, p, requests, width, p, 9, head, shares, layers, 2, 64, blocks, block, p, p, p,
                        None)
    assert fork(src=None) == -1 and fork(lens=None) == -1 and fork(shares=None) == -1 and fork(head=None) == -1
    assert fork(forks=8193) == -2 and fork(requests=8193) == -2 and fork(layers=0) == -2 and fork(block=2048) == -2
    free = lambda rows=p, count=2, lens=p, requests=3, shares=p, blocks=64, block=16, ws=p, size=1 << 20: L.dgt_page_free(
        rows, count, lens, p, requests, 4, p, 9, p, shares, blocks, block, p, ws, size, None)
    assert free(rows=None) == -1 and free(lens=None) == -1 and free(shares=None) == -1 and free(ws=None) == -1
    assert free(ws=258) == -1 and free(count=8193) == -2 and free(block=3) == -2
    assert free(size=dgt.dgt_page_free_workspace(64) - 1) == -4


def test_empty_calls_do_nothing():
    """No token: success without a launch (the pointers are never read)."""
    L = dgt.lib()
    assert L.dgt_rope_store(None, None, None, 3, 0, 0, 0, 0, 0, 0, None, None, 0, 4, 2, 64, None, 32, 0, None, None, 1e-6, 1,
                            None, 0, 0, None, None, 8, 16, None) == 0
    assert L.dgt_chunk_attention(1, None, 0, 0, None, None, 8, 16, None, 4, None, None, 2, 0, 4, 2, 64, 0.1, None, 0, 0,
                                 None, 0, None) == 0
    assert L.dgt_verify(3, None, 50, None, None, 0, None, None, None, None, None, 0, 0, 50, None, None, None, None, 0,
                        None) == 0


def test_more_work_than_a_launch_counts():
    """Workgroups past 2^24 of 256 threads are refused before anything is launched."""
    L, p = dgt.lib(), 256
    assert L.dgt_rope_store(p, p, p, 3, 65536, 8, 65536, 8, 65536, 8, p, p, 1 << 17, 8192, 8192, 8, None, 0, 0, None, None,
                            1e-6, 1, p, 65536, 8, p, p, 8, 16, None) == -2
    assert L.dgt_verify_workspace(1 << 15, 1 << 21, 4) == 0 and L.dgt_verify_workspace((1 << 15) - 1, 1 << 21, 4) > 0
    assert L.dgt_verify(3, p, 1 << 21, p, None, 0, None, p, None, p, p, 4, 1 << 15, 1 << 21, p, p, p, p, 1 << 40, None) == -2
