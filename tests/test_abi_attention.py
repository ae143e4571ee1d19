"""Host-side checks of rotary positions, the cache append and attention (CPU
only): every refusal happens before a device is touched, with the documented
status."""
import ctypes
import math

import pytest

import gguf_block_quant_qmm_amd as q

A = 0x7F0000000000  # a 16-byte aligned fake device address: never dereferenced
BIG = 1 << 40


def rope(X=A, x_stride=0, N=3, H=4, D=64, pos=A, freqs=A, rot=32, layout=1, mscale=1.0, Y=A, y_stride=0):
    return q.lib().qmm_rope(X, x_stride, N, H, D, pos, freqs, rot, layout, mscale, Y, y_stride, None)


@pytest.mark.parametrize("kw,code", [
    (dict(N=0), q.QMM_ERR_SHAPE), (dict(N=1 << 31), q.QMM_ERR_SHAPE), (dict(H=0), q.QMM_ERR_SHAPE),
    (dict(H=65537), q.QMM_ERR_SHAPE), (dict(D=60), q.QMM_ERR_SHAPE), (dict(D=1032, rot=8), q.QMM_ERR_SHAPE),
    (dict(rot=0), q.QMM_ERR_SHAPE), (dict(rot=12), q.QMM_ERR_SHAPE), (dict(rot=72), q.QMM_ERR_SHAPE),
    (dict(x_stride=252), q.QMM_ERR_SHAPE), (dict(x_stride=258), q.QMM_ERR_SHAPE), (dict(x_stride=-256), q.QMM_ERR_SHAPE),
    (dict(y_stride=255), q.QMM_ERR_SHAPE), (dict(y_stride=BIG + 4), q.QMM_ERR_SHAPE),
    (dict(layout=2), q.QMM_ERR_VALUE), (dict(layout=-1), q.QMM_ERR_VALUE), (dict(mscale=math.nan), q.QMM_ERR_VALUE),
    (dict(X=0), q.QMM_ERR_NULL), (dict(pos=0), q.QMM_ERR_NULL), (dict(freqs=0), q.QMM_ERR_NULL), (dict(Y=0), q.QMM_ERR_NULL),
    (dict(X=A + 4), q.QMM_ERR_ALIGN), (dict(Y=A + 8), q.QMM_ERR_ALIGN), (dict(pos=A + 2), q.QMM_ERR_ALIGN),
    (dict(freqs=A + 1), q.QMM_ERR_ALIGN),
])
def test_rope_rejects(kw, code):
    assert rope(**kw) == code


def freqs(rot=64, base=1e4, factor=1.0, context=0.0, fast=32.0, slow=1.0, factors=0, out=A):
    return q.lib().qmm_rope_freqs(rot, base, factor, context, fast, slow, factors, out, None)


@pytest.mark.parametrize("kw,code", [
    (dict(rot=0), q.QMM_ERR_SHAPE), (dict(rot=7), q.QMM_ERR_SHAPE), (dict(rot=1026), q.QMM_ERR_SHAPE),
    (dict(base=1.0), q.QMM_ERR_VALUE), (dict(base=math.inf), q.QMM_ERR_VALUE), (dict(factor=0.0), q.QMM_ERR_VALUE),
    (dict(context=-1.0), q.QMM_ERR_VALUE), (dict(slow=0.0), q.QMM_ERR_VALUE), (dict(fast=1.0), q.QMM_ERR_VALUE),
    (dict(factor=math.nan), q.QMM_ERR_VALUE), (dict(out=0), q.QMM_ERR_NULL), (dict(factors=A + 2), q.QMM_ERR_ALIGN),
])
def test_rope_freqs_rejects(kw, code):
    assert freqs(**kw) == code


CACHE = dict(k=A, v=A, pages=10, dtype=1, page=64, heads=4, dim=128)
BATCH = dict(table=A, lens=A, starts=0, seqs=3, max_pages=8, table_stride=0, max_new=2, rows=6)


def structs(kw):
    """(cache, batch, the other arguments) of kw."""
    c, b = ({k: kw.get(k, v) for k, v in d.items()} for d in (CACHE, BATCH))
    rest = {k: v for k, v in kw.items() if k not in CACHE and k not in BATCH}
    return q._KvCacheStruct(*(c[k] for k, _ in q._KvCacheStruct._fields_)), q._KvBatchStruct(
        *(b[k] for k, _ in q._KvBatchStruct._fields_)), rest


def append(K=A, k_stride=0, V=A, v_stride=0, freqs=A, rot=128, layout=0, mscale=1.0, pos=0, k_norm=0, q_norm=0, eps=1e-5,
           Q=A, q_stride=0, q_heads=8, q_out=A, no_cache=False, no_batch=False, **kw):
    c, b, rest = structs(kw)
    assert not rest
    return q.lib().qmm_kv_append(None if no_cache else ctypes.addressof(c), None if no_batch else ctypes.addressof(b), K,
                                 k_stride, V, v_stride, freqs, rot, layout, mscale, pos, k_norm, q_norm, eps, Q, q_stride,
                                 q_heads, q_out, None)


SIZES = [
    (dict(dtype=0), q.QMM_ERR_DTYPE), (dict(dtype=2), q.QMM_ERR_DTYPE), (dict(pages=0), q.QMM_ERR_SHAPE),
    (dict(pages=1 << 31), q.QMM_ERR_SHAPE), (dict(page=8), q.QMM_ERR_SHAPE), (dict(page=48), q.QMM_ERR_SHAPE),
    (dict(page=2048), q.QMM_ERR_SHAPE), (dict(heads=0), q.QMM_ERR_SHAPE), (dict(heads=1025), q.QMM_ERR_SHAPE),
    (dict(dim=32), q.QMM_ERR_SHAPE), (dict(dim=80), q.QMM_ERR_SHAPE), (dict(dim=512), q.QMM_ERR_SHAPE),
    (dict(seqs=0), q.QMM_ERR_SHAPE), (dict(seqs=65536, rows=1 << 20), q.QMM_ERR_SHAPE), (dict(max_new=0), q.QMM_ERR_SHAPE),
    (dict(seqs=2, max_new=1 << 30, rows=1 << 30), q.QMM_ERR_SHAPE), (dict(rows=0), q.QMM_ERR_SHAPE),
    (dict(rows=5), q.QMM_ERR_SHAPE), (dict(rows=1 << 31), q.QMM_ERR_SHAPE), (dict(max_pages=0), q.QMM_ERR_SHAPE),
    (dict(max_pages=1 << 25), q.QMM_ERR_SHAPE), (dict(table_stride=7), q.QMM_ERR_SHAPE),
    (dict(table_stride=-8), q.QMM_ERR_SHAPE), (dict(no_cache=True), q.QMM_ERR_NULL), (dict(no_batch=True), q.QMM_ERR_NULL),
    (dict(k=0), q.QMM_ERR_NULL), (dict(v=0), q.QMM_ERR_NULL), (dict(table=0), q.QMM_ERR_NULL), (dict(lens=0), q.QMM_ERR_NULL),
    (dict(k=A + 8), q.QMM_ERR_ALIGN), (dict(v=A + 2), q.QMM_ERR_ALIGN), (dict(table=A + 2), q.QMM_ERR_ALIGN),
    (dict(lens=A + 1), q.QMM_ERR_ALIGN), (dict(starts=A + 2), q.QMM_ERR_ALIGN),
]


@pytest.mark.parametrize("kw,code", SIZES + [
    (dict(k_stride=508), q.QMM_ERR_SHAPE), (dict(v_stride=514), q.QMM_ERR_SHAPE), (dict(q_stride=1000), q.QMM_ERR_SHAPE),
    (dict(rot=12), q.QMM_ERR_SHAPE), (dict(rot=136), q.QMM_ERR_SHAPE), (dict(rot=0), q.QMM_ERR_SHAPE),
    (dict(q_heads=0), q.QMM_ERR_SHAPE), (dict(q_heads=65537), q.QMM_ERR_SHAPE), (dict(layout=3), q.QMM_ERR_VALUE),
    (dict(mscale=math.inf), q.QMM_ERR_VALUE), (dict(eps=-1.0), q.QMM_ERR_VALUE), (dict(eps=math.nan), q.QMM_ERR_VALUE),
    (dict(K=0), q.QMM_ERR_NULL), (dict(V=0), q.QMM_ERR_NULL), (dict(Q=0), q.QMM_ERR_NULL), (dict(q_out=0), q.QMM_ERR_NULL),
    (dict(K=A + 4), q.QMM_ERR_ALIGN), (dict(V=A + 8), q.QMM_ERR_ALIGN), (dict(Q=A + 4), q.QMM_ERR_ALIGN),
    (dict(q_out=A + 4), q.QMM_ERR_ALIGN), (dict(k_norm=A + 4), q.QMM_ERR_ALIGN), (dict(q_norm=A + 8), q.QMM_ERR_ALIGN),
    (dict(freqs=A + 2), q.QMM_ERR_ALIGN), (dict(pos=A + 1), q.QMM_ERR_ALIGN),
])
def test_kv_append_rejects(kw, code):
    assert append(**kw) == code


def attention(Q=A, q_stride=0, q_heads=8, scale=0.1, causal=1, window=0, softcap=0.0, out=A, work=A, work_bytes=BIG,
              no_cache=False, no_batch=False, **kw):
    c, b, rest = structs(kw)
    assert not rest
    return q.lib().qmm_attention(None if no_cache else ctypes.addressof(c), None if no_batch else ctypes.addressof(b), Q,
                                 q_stride, q_heads, scale, causal, window, softcap, out, work, work_bytes, None)


@pytest.mark.parametrize("kw,code", SIZES + [
    (dict(q_heads=0), q.QMM_ERR_SHAPE), (dict(q_heads=2), q.QMM_ERR_SHAPE), (dict(q_heads=10), q.QMM_ERR_SHAPE),
    (dict(q_heads=65540), q.QMM_ERR_SHAPE), (dict(q_stride=1020), q.QMM_ERR_SHAPE), (dict(q_stride=1026), q.QMM_ERR_SHAPE),
    (dict(heads=1, q_heads=64, seqs=1, max_new=1 << 26, rows=1 << 26), q.QMM_ERR_SHAPE),
    (dict(rows=(1 << 31) - 1, starts=A, q_heads=1024), q.QMM_ERR_SHAPE),
    (dict(scale=math.nan), q.QMM_ERR_VALUE), (dict(scale=1e300), q.QMM_ERR_VALUE), (dict(softcap=-1.0), q.QMM_ERR_VALUE),
    (dict(softcap=math.inf), q.QMM_ERR_VALUE), (dict(window=-1), q.QMM_ERR_VALUE),
    (dict(window=5, causal=0), q.QMM_ERR_VALUE), (dict(Q=0), q.QMM_ERR_NULL), (dict(out=0), q.QMM_ERR_NULL),
    (dict(Q=A + 4), q.QMM_ERR_ALIGN), (dict(out=A + 8), q.QMM_ERR_ALIGN),
])
def test_attention_rejects(kw, code):
    assert attention(**kw) == code


def test_attention_work_is_checked():
    kw = dict(max_pages=1000, pages=4000)
    c, b, _ = structs(kw)
    n = q.lib().qmm_attention_work_bytes(ctypes.addressof(c), ctypes.addressof(b), 8)
    assert n > 0
    assert attention(work=0, work_bytes=0, **kw) == q.QMM_ERR_NULL
    assert attention(work=A + 8, work_bytes=n, **kw) == q.QMM_ERR_ALIGN
    assert attention(work=A, work_bytes=n - 1, **kw) == q.QMM_ERR_SCRATCH
    for bad in (dict(dtype=3), dict(seqs=0), dict(dim=80)):
        c, b, _ = structs(bad)
        assert q.lib().qmm_attention_work_bytes(ctypes.addressof(c), ctypes.addressof(b), 8) == 0
    assert q.lib().qmm_attention_work_bytes(None, ctypes.addressof(b), 8) == 0


def test_pool_bytes():
    assert q.kv_pool_bytes(1, 10, 64, 8, 128) == 10 * 64 * 8 * 128 * 2
    assert q.kv_pool_bytes(8, 10, 64, 8, 128) == 10 * 64 * 8 * (128 + 8)
    assert q.kv_pool_bytes(1, 1 << 30, 1024, 1024, 256) == 1 << 59
    assert q.kv_pool_bytes(2, 10, 64, 8, 128) == 0 and q.kv_pool_bytes(1, 10, 24, 8, 128) == 0
    assert q.kv_pool_bytes(1, 10, 64, 8, 100) == 0 and q.kv_pool_bytes(1, 0, 64, 8, 128) == 0


def test_valid_calls_without_gpu_report_device():
    import torch
    if torch.cuda.is_available():
        pytest.skip("a GPU is present; covered by the GPU tests")
    assert rope() == q.QMM_ERR_DEVICE and freqs() == q.QMM_ERR_DEVICE and append() == q.QMM_ERR_DEVICE
    assert attention() == q.QMM_ERR_DEVICE and attention(causal=0, starts=A, rows=1, dtype=8) == q.QMM_ERR_DEVICE
    assert append(Q=0, q_out=0, q_heads=0, freqs=0, rot=0, layout=9, dtype=8, starts=A, rows=1) == q.QMM_ERR_DEVICE


@pytest.mark.parametrize("kw,code", [
    (dict(page=(1 << 32) + 64), q.QMM_ERR_SHAPE), (dict(heads=(1 << 32) + 4), q.QMM_ERR_SHAPE),
    (dict(dim=(1 << 32) + 128), q.QMM_ERR_SHAPE), (dict(pages=0), q.QMM_ERR_SHAPE), (dict(dtype=2), q.QMM_ERR_DTYPE),
])
def test_cache_description_refuses_what_its_fields_would_cut(kw, code):
    with pytest.raises(q.QmmError) as e:
        q.KvCache(A, A, **{**dict(dtype=1, pages=10, page=64, heads=4, dim=128), **kw})
    assert e.value.code == code


@pytest.mark.parametrize("kw", [dict(seqs=-1), dict(rows=1 << 64), dict(max_pages=1 << 63), dict(max_new=-2)])
def test_batch_description_refuses_what_its_fields_would_cut(kw):
    with pytest.raises(q.QmmError) as e:
        q.KvBatch(A, A, **{**dict(seqs=3, max_pages=8, max_new=2, rows=6), **kw})
    assert e.value.code == q.QMM_ERR_SHAPE


def test_host_tensors_are_refused():
    import torch
    with pytest.raises(ValueError, match="device"):
        q.KvCache(torch.zeros(q.kv_pool_bytes(1, 2, 16, 1, 64), dtype=torch.uint8), A, 1, 2, 16, 1, 64)
    with pytest.raises(ValueError, match="device"):
        q.KvBatch(torch.zeros(4, dtype=torch.int32), A, 1, 4, 1, 1)
