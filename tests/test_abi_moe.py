"""Host-side checks of the sparse feed-forward block's calls (CPU only): every
refusal happens before a device is touched, with the documented status."""
import ctypes
import math

import pytest

import gguf_block_quant_qmm_amd as q

A = 0x7F0000000000  # a 16-byte aligned fake device address: never dereferenced
BIG = 1 << 40


def norm(block=A, w_post=A, gate=A, gate_stride=0, scale=1.0, residual=A, residual_out=A, w_pre=A, eps=1e-5, N=3, K=64,
         H=A, scales=A, quants=A):
    return q.lib().qmm_block_norm(block, w_post, gate, gate_stride, scale, residual, residual_out, w_pre, eps, N, K, H,
                                  scales, quants, None)


@pytest.mark.parametrize("kw,code", [
    (dict(N=0), q.QMM_ERR_SHAPE), (dict(N=1 << 31), q.QMM_ERR_SHAPE), (dict(K=0), q.QMM_ERR_SHAPE),
    (dict(K=(1 << 28) + 32), q.QMM_ERR_SHAPE), (dict(gate_stride=32), q.QMM_ERR_SHAPE),
    (dict(gate_stride=-64), q.QMM_ERR_SHAPE), (dict(K=48), q.QMM_ERR_SHAPE), (dict(K=33), q.QMM_ERR_SHAPE),
    (dict(scale=math.inf), q.QMM_ERR_VALUE), (dict(scale=math.nan), q.QMM_ERR_VALUE),
    (dict(eps=-1e-6), q.QMM_ERR_VALUE), (dict(eps=math.nan), q.QMM_ERR_VALUE), (dict(eps=math.inf), q.QMM_ERR_VALUE),
    (dict(residual=0), q.QMM_ERR_NULL), (dict(residual_out=0), q.QMM_ERR_NULL), (dict(scales=0), q.QMM_ERR_NULL),
    (dict(quants=0), q.QMM_ERR_NULL), (dict(block=0, residual_out=0, H=0, scales=0, quants=0), q.QMM_ERR_NULL),
    (dict(block=A + 4), q.QMM_ERR_ALIGN), (dict(residual=A + 8), q.QMM_ERR_ALIGN), (dict(w_pre=A + 4), q.QMM_ERR_ALIGN),
    (dict(H=A + 4), q.QMM_ERR_ALIGN), (dict(quants=A + 1), q.QMM_ERR_ALIGN), (dict(scales=A + 4), q.QMM_ERR_ALIGN),
    (dict(gate=A + 4), q.QMM_ERR_ALIGN), (dict(w_post=A + 4), q.QMM_ERR_ALIGN), (dict(residual_out=A + 4), q.QMM_ERR_ALIGN),
])
def test_block_norm_rejects(kw, code):
    assert norm(**kw) == code


def route(logits=A, bias=A, N=3, E=64, scoring=0, groups=8, topk_groups=4, group_top=2, topk=8, renorm=1, scale=1.0, ids=A,
          weights=A):
    return q.lib().qmm_moe_route(logits, bias, N, E, scoring, groups, topk_groups, group_top, topk, renorm, scale, ids,
                                 weights, None)


@pytest.mark.parametrize("kw,code", [
    (dict(N=0), q.QMM_ERR_SHAPE), (dict(N=1 << 31), q.QMM_ERR_SHAPE), (dict(E=0), q.QMM_ERR_SHAPE),
    (dict(E=1032), q.QMM_ERR_SHAPE), (dict(groups=0), q.QMM_ERR_SHAPE), (dict(groups=7), q.QMM_ERR_SHAPE),
    (dict(groups=128), q.QMM_ERR_SHAPE), (dict(topk_groups=0), q.QMM_ERR_SHAPE), (dict(topk_groups=9), q.QMM_ERR_SHAPE),
    (dict(group_top=0), q.QMM_ERR_SHAPE), (dict(group_top=3), q.QMM_ERR_SHAPE),
    (dict(groups=64, topk_groups=64, group_top=2), q.QMM_ERR_SHAPE), (dict(topk=0), q.QMM_ERR_SHAPE),
    (dict(topk=33, topk_groups=8), q.QMM_ERR_SHAPE), (dict(topk=9, topk_groups=1), q.QMM_ERR_SHAPE),
    (dict(scoring=2), q.QMM_ERR_VALUE), (dict(scoring=-1), q.QMM_ERR_VALUE), (dict(scale=math.nan), q.QMM_ERR_VALUE),
    (dict(logits=0), q.QMM_ERR_NULL), (dict(ids=0), q.QMM_ERR_NULL), (dict(weights=0), q.QMM_ERR_NULL),
    (dict(logits=A + 2), q.QMM_ERR_ALIGN), (dict(bias=A + 1), q.QMM_ERR_ALIGN), (dict(ids=A + 2), q.QMM_ERR_ALIGN),
    (dict(weights=A + 3), q.QMM_ERR_ALIGN),
])
def test_moe_route_rejects(kw, code):
    assert route(**kw) == code


def swiglu(gate=A, up=A, dtype=2, E=8, M=64, K=256, N=64, T=2, ids=A, X=A, out=A, work=A, work_bytes=BIG):
    return q.lib().qmm_moe_swiglu(gate, up, dtype, E, M, K, N, T, ids, X, out, work, work_bytes, None)


def down(w=A, dtype=2, E=8, M=64, K=256, N=64, T=2, ids=A, weights=A, H=A, residual=A, Y=A, work=A, work_bytes=BIG):
    return q.lib().qmm_moe_down(w, dtype, E, M, K, N, T, ids, weights, H, residual, Y, work, work_bytes, None)


SIZES = [
    (dict(dtype=5), q.QMM_ERR_DTYPE), (dict(M=0), q.QMM_ERR_SHAPE), (dict(K=48), q.QMM_ERR_SHAPE),
    (dict(dtype=14, K=128), q.QMM_ERR_SHAPE), (dict(N=0), q.QMM_ERR_SHAPE), (dict(E=0), q.QMM_ERR_SHAPE),
    (dict(E=1025), q.QMM_ERR_SHAPE), (dict(T=0), q.QMM_ERR_SHAPE), (dict(T=33), q.QMM_ERR_SHAPE),
    (dict(N=1 << 30, T=2), q.QMM_ERR_SHAPE), (dict(E=1024, M=1 << 28, K=1 << 20, N=1), q.QMM_ERR_SHAPE),
    (dict(M=1 << 39, K=32, N=1 << 16, T=8), q.QMM_ERR_SHAPE), (dict(N=-1), q.QMM_ERR_SHAPE),
]


@pytest.mark.parametrize("kw,code", SIZES + [
    (dict(gate=0), q.QMM_ERR_NULL), (dict(up=0), q.QMM_ERR_NULL), (dict(ids=0), q.QMM_ERR_NULL),
    (dict(X=0), q.QMM_ERR_NULL), (dict(out=0), q.QMM_ERR_NULL), (dict(gate=A + 8), q.QMM_ERR_ALIGN),
    (dict(up=A + 2), q.QMM_ERR_ALIGN), (dict(X=A + 4), q.QMM_ERR_ALIGN), (dict(ids=A + 2), q.QMM_ERR_ALIGN),
    (dict(out=A + 2), q.QMM_ERR_ALIGN),
])
def test_moe_swiglu_rejects(kw, code):
    assert swiglu(**kw) == code


@pytest.mark.parametrize("kw,code", SIZES + [
    (dict(w=0), q.QMM_ERR_NULL), (dict(weights=0), q.QMM_ERR_NULL), (dict(ids=0), q.QMM_ERR_NULL),
    (dict(H=0), q.QMM_ERR_NULL), (dict(Y=0), q.QMM_ERR_NULL), (dict(w=A + 8), q.QMM_ERR_ALIGN),
    (dict(H=A + 4), q.QMM_ERR_ALIGN), (dict(weights=A + 2), q.QMM_ERR_ALIGN), (dict(residual=A + 1), q.QMM_ERR_ALIGN),
    (dict(Y=A + 2), q.QMM_ERR_ALIGN),
])
def test_moe_down_rejects(kw, code):
    assert down(**kw) == code


@pytest.mark.parametrize("call,need", [(swiglu, q.moe_swiglu_work_bytes), (down, q.moe_down_work_bytes)])
@pytest.mark.parametrize("dims,some", [((2, 8, 1024, 4096, 512, 2), True), ((14, 64, 1024, 2048, 512, 8), True),
                                       ((8, 4, 63, 96, 3, 1), False), ((12, 8, 14336, 4096, 1, 2), False)])
def test_moe_work_is_checked(call, need, dims, some):
    dtype, E, M, K, N, T = dims
    kw = dict(dtype=dtype, E=E, M=M, K=K, N=N, T=T)
    n = need(*dims)
    assert (n > 0) == some  # few tokens need no workspace
    if n:
        assert call(work=0, work_bytes=0, **kw) == q.QMM_ERR_NULL
        assert call(work=A + 8, work_bytes=n, **kw) == q.QMM_ERR_ALIGN
        assert call(work=A, work_bytes=n - 1, **kw) == q.QMM_ERR_SCRATCH


def test_work_bytes_of_bad_sizes_are_zero():
    for need in (q.moe_swiglu_work_bytes, q.moe_down_work_bytes):
        assert need(5, 8, 64, 256, 64, 2) == 0
        assert need(2, 0, 64, 256, 64, 2) == 0
        assert need(2, 8, 64, 48, 64, 2) == 0
        assert need(2, 8, 64, 256, 64, 64) == 0


def test_valid_calls_without_gpu_report_device():
    import torch
    if torch.cuda.is_available():
        pytest.skip("a GPU is present; covered by the GPU tests")
    assert norm() == q.QMM_ERR_DEVICE
    assert norm(block=0, residual_out=0, quants=0, scales=0, K=33) == q.QMM_ERR_DEVICE
    assert route() == q.QMM_ERR_DEVICE
    assert route(bias=0, groups=1, topk_groups=1, group_top=1) == q.QMM_ERR_DEVICE
    assert swiglu() == q.QMM_ERR_DEVICE
    assert down(residual=0) == q.QMM_ERR_DEVICE


def test_strerror_names_the_value_status():
    assert "range" in q.strerror(q.QMM_ERR_VALUE) and ctypes.c_char_p(q.strerror(-7).encode()).value


def test_work_without_a_size_is_refused():
    for call, rest in ((q.qmm_moe_swiglu, (A, A, 2, 8, 64, 256, 64, 2, A, A, A)), (q.qmm_moe_down, (A, 2, 8, 64, 256, 64, 2, A, A, A, A))):
        with pytest.raises(ValueError, match="work"):
            call(*rest, work=A)
