"""Refusals of the paged KV cache's entry points, without a GPU: each is found
on the host before anything is launched."""
import ctypes

import pytest
import torch

import mixed_bitwidth_weight_b200 as q

A = 0x7f0000000000  # never dereferenced
OK, NULL, SHAPE, BITS, ALIGN, WS, DTYPE = 0, -1, -2, -3, -4, -5, -6


def cache(**kw):
    a = dict(d_pages=A, num_pages=4, page_size=64, kv_heads=2, head_dim=128, k_bits=4, v_bits=4)
    a.update(kw)
    return q._CacheStruct(**a)


def batch(**kw):
    a = dict(d_block_table=A, table_stride=8, d_seq_lens=A, d_cu_new=A, num_seqs=3, max_pages=8)
    a.update(kw)
    return q._BatchStruct(**a)


def move(fn, c=None, b=None, rows=5, k=A, krs=256, khs=128, v=A, vrs=256, vhs=128, dt=0):
    c, b = c or cache(), b or batch()
    return fn(ctypes.byref(c), ctypes.byref(b), rows, k, krs, khs, v, vrs, vhs, dt, None)


def attend(c=None, b=None, rows=5, qp=A, qrs=1024, qhs=128, dt=0, heads=8, scale=0.1, window=0, out=A, ors=1024,
           ohs=128, lse=A, ws=A, wsb=None):
    c, b = c or cache(), b or batch()
    if wsb is None:
        wsb = q._lib.qgemm_kv_attend_workspace_bytes(ctypes.byref(c), heads)
    return q._lib.qgemm_kv_attend(ctypes.byref(c), ctypes.byref(b), rows, qp, qrs, qhs, dt, heads, scale, window, out,
                                  ors, ohs, lse, ws, wsb, None)


BAD_CACHE = [(dict(d_pages=0), NULL), (dict(num_pages=0), SHAPE), (dict(num_pages=1 << 31), SHAPE),
             (dict(page_size=16), SHAPE), (dict(page_size=96), SHAPE), (dict(kv_heads=0), SHAPE),
             (dict(head_dim=32), SHAPE), (dict(head_dim=192), SHAPE), (dict(k_bits=7), BITS), (dict(v_bits=1), BITS),
             (dict(d_pages=A + 64), ALIGN)]
BAD_BATCH = [(dict(num_seqs=-1), SHAPE), (dict(num_seqs=65536), SHAPE), (dict(max_pages=-1), SHAPE),
             (dict(table_stride=7), SHAPE), (dict(d_block_table=0), NULL), (dict(d_seq_lens=0), NULL),
             (dict(d_cu_new=0), NULL), (dict(d_seq_lens=A + 2), ALIGN)]


def entries():
    lib = q._lib
    return [lambda **kw: move(lib.qgemm_kv_append, **kw), lambda **kw: move(lib.qgemm_kv_gather, **kw), attend]


@pytest.mark.parametrize("n", range(3))
def test_bad_caches_and_batches(n):
    fn = entries()[n]
    for kw, status in BAD_CACHE:
        extra = dict(wsb=1 << 30) if n == 2 else {}
        assert fn(c=cache(**kw), **extra) == status, kw
    for kw, status in BAD_BATCH:
        assert fn(b=batch(**kw)) == status, kw
    assert fn(rows=-1) == SHAPE
    assert fn(dt=2) == DTYPE
    assert fn(b=batch(num_seqs=0, d_block_table=0, d_seq_lens=0, d_cu_new=0)) == OK     # nothing to do
    assert fn(rows=0) == OK


def test_move_operands():
    lib = q._lib
    for fn in (lib.qgemm_kv_append, lib.qgemm_kv_gather):
        assert move(fn, k=0) == NULL
        assert move(fn, v=0) == NULL
        assert move(fn, k=A + 8) == ALIGN
        assert move(fn, krs=260) == ALIGN
        assert move(fn, vhs=130) == ALIGN
        assert move(fn, krs=-256) == SHAPE
    # a written operand may not overlap itself; a read one may (an expanded view)
    assert move(lib.qgemm_kv_gather, krs=128) == SHAPE
    assert move(lib.qgemm_kv_gather, khs=0) == SHAPE
    assert move(lib.qgemm_kv_gather, vrs=0) == SHAPE


def test_attend_operands():
    assert attend(qp=0) == NULL
    assert attend(out=0) == NULL
    assert attend(heads=7) == SHAPE
    assert attend(heads=0, wsb=1 << 20) == SHAPE
    assert attend(window=-1) == SHAPE
    assert attend(scale=float("nan")) == SHAPE
    assert attend(scale=float("inf")) == SHAPE
    assert attend(ws=0) == WS
    assert attend(wsb=8) == WS
    assert attend(ws=A + 4) == ALIGN
    assert attend(lse=A + 2) == ALIGN
    assert attend(qp=A + 2) == ALIGN
    assert attend(ors=512) == SHAPE
    assert attend(ohs=0) == SHAPE


def test_workspace_size():
    c = cache()
    f = q._lib.qgemm_kv_attend_workspace_bytes
    assert f(ctypes.byref(c), 8) > 0
    assert f(ctypes.byref(c), 9) == 0 and f(ctypes.byref(c), 0) == 0 and f(None, 8) == 0
    assert f(ctypes.byref(cache(head_dim=80)), 8) == 0


def test_binding_refuses_before_the_library():
    words = q.qgemm_kv_page_words(2, 128, 4, 4, 64)
    with pytest.raises(TypeError):
        q.KVCache(torch.zeros(3, words, dtype=torch.int32), 64, 2, 128, 4, 4)            # a host tensor
    with pytest.raises(ValueError):
        q.KVCache(torch.zeros(3, words - 1, dtype=torch.int32), 64, 2, 128, 4, 4)
    with pytest.raises(q.QGemmError):
        q.KVCache(torch.zeros(3, words, dtype=torch.int32), 60, 2, 128, 4, 4)
    t, l, cu = (torch.zeros(*s, dtype=torch.int32) for s in ((2, 4), (2,), (3,)))
    with pytest.raises(TypeError):
        q.KVBatch(t, l, cu)
    with pytest.raises(ValueError):
        q.KVBatch(t, l, cu[:2])
    with pytest.raises(ValueError):
        q.KVBatch(t[0], l, cu)
