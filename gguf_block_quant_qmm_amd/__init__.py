"""Python binding of libqmm, the GGUF block-quantized matmul for MI355X.

Argument marshalling only: every step of the computation runs in the HIP
kernels behind the C ABI of include/qmm.h.  Tensors are PyTorch device
tensors (PyTorch supplies device memory and streams); the functions also
accept raw device addresses as ints.  If libqmm.so is missing the calls raise;
there is no CPU fallback.

    qmm_gemv(w, dtype, M, K, x, y, stream=None)      y[M] = W x
    qmm_gemm(w, dtype, M, K, N, X, Y, stream=None)   Y[N][M] = X W^T
    qmm_gemv_concat(ws, dtype, Ms, K, x, ys, stream=None)
                                                     ys[i] = W_i x, one launch
    qmm_gemv_swiglu(gate, up, dtype, M, K, x, out, stream=None)
                                                     out = silu(W_gate x) * (W_up x)
    qmm_gemv_argmax(w, dtype, M, K, x, work, index, value=None, stream=None)
                                                     index = argmax_m (W x)[m]
    qmm_gemv_argmax_noalloc(w, dtype, M, K, x, index, value=None, stream=None)
                                                     the same, scratch in a static
                                                     device array (no work buffer)
    qmm_gemm_swiglu(gate, up, dtype, M, K, N, X, out, stream=None)
                                                     out = silu(X Wg^T) * (X Wu^T)
    qmm_quantize_q8_0(X, N, K, scales, quants, stream=None)
                                                     X -> Q8_0 activation blocks
    qmm_gemm_q8act(w, dtype, M, K, N, scales, quants, Y, stream=None)
                                                     Y = Xq W^T (int8 activations)
    qmm_repack(w, dtype, M, K, packed, stream=None)  Q6_K / Q8_0 -> the GEMM's repacked layout
    qmm_gemm_repacked(packed, dtype, M, K, N, X, Y, stream=None)
                                                     Y[N][M] = X W^T from the repacked copy
    qmm_gemv_q8act / qmm_gemv_concat_q8act / qmm_gemv_swiglu_q8act /
    qmm_gemv_argmax_q8act                            the decode calls above with x
                                                     quantized inside the launch
    qmm_block_norm(residual, N, K, residual_out=None, block=None, w_post=None, gate=None,
                   gate_stride=0, scale=1.0, w_pre=None, eps=1e-5, H=None, scales=None,
                   quants=None, stream=None)         the norms after and before a block with
                                                     its gate and residual scale
    qmm_moe_route(logits, N, E, topk, ids, weights, bias=None, scoring=QMM_ROUTE_SOFTMAX,
                  groups=1, topk_groups=1, group_top=1, renorm=True, scale=1.0, stream=None)
                                                     each token's topk experts and weights
    qmm_moe_swiglu(gate, up, dtype, E, M, K, N, T, ids, X, out, work=None, stream=None)
                                                     out[n][t] = silu(G_e x_n) * (U_e x_n)
    qmm_moe_down(w, dtype, E, M, K, N, T, ids, weights, H, Y, residual=None, work=None,
                 stream=None)                        Y[n] = residual[n] + sum_t w_nt W_e h_nt
    qmm_rope_freqs(rot, base, freqs, factor=1.0, context=0.0, beta_fast=32.0, beta_slow=1.0,
                   factors=None, stream=None)        frequencies: plain, linear, YaRN, per pair
    qmm_rope(X, N, H, D, pos, freqs, rot, Y, layout=QMM_ROPE_HALF, mscale=1.0, x_stride=0,
             y_stride=0, stream=None)                heads turned by their token's position
    KvCache(k, v, dtype, pages, page, heads, dim)    a paged key-value cache (f16 or Q8_0 pools)
    KvBatch(table, lens, seqs, max_pages, max_new, rows, starts=None, table_stride=0)
                                                     a call's sequences and their new tokens
    qmm_kv_append(cache, batch, K, V, freqs=None, rot=0, layout=QMM_ROPE_HALF, mscale=1.0,
                  pos=None, k_norm=None, q_norm=None, eps=1e-5, Q=None, q_heads=0, q_out=None,
                  q_stride=0, k_stride=0, v_stride=0, stream=None)
                                                     keys (turned) and values into the cache,
                                                     the queries turned beside them
    qmm_attention(cache, batch, Q, q_heads, out, scale=None, causal=True, window=0, softcap=0.0,
                  work=None, q_stride=0, stream=None)
                                                     the new tokens' attention over the cache
"""
from __future__ import annotations

import ctypes
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libqmm.so")

# dtype tags (GGUF type ids) and status codes, as in include/qmm.h
QMM_Q4_0, QMM_Q4_1, QMM_Q8_0, QMM_Q4_K, QMM_Q5_K, QMM_Q6_K = 2, 3, 8, 12, 13, 14
DTYPES = {"Q4_0": QMM_Q4_0, "Q4_1": QMM_Q4_1, "Q8_0": QMM_Q8_0, "Q4_K": QMM_Q4_K, "Q5_K": QMM_Q5_K,
          "Q6_K": QMM_Q6_K}
QMM_OK, QMM_ERR_NULL, QMM_ERR_DTYPE, QMM_ERR_SHAPE = 0, -1, -2, -3
QMM_ERR_ALIGN, QMM_ERR_DEVICE, QMM_ERR_LAUNCH, QMM_ERR_SCRATCH, QMM_ERR_VALUE = -4, -5, -6, -7, -8

QMM_GEMV_MAX_MATS = 4
QMM_ARGMAX_WORK_BYTES = 32768
QMM_NOALLOC_SCRATCH_BYTES = 32768
QMM_READ_PROBE_OUT_FLOATS = 4096
QMM_ROUTE_SOFTMAX, QMM_ROUTE_SIGMOID = 0, 1
QMM_F16 = 1
QMM_ROPE_INTERLEAVED, QMM_ROPE_HALF = 0, 1
QMM_MOE_MAX_EXPERTS, QMM_MOE_MAX_TOPK, QMM_MOE_MAX_ROWS, QMM_MOE_MAX_K = 1024, 32, 4194304, 1048576

EXPORTS = ("qmm_gemv", "qmm_gemv_concat", "qmm_gemv_swiglu", "qmm_gemv_argmax", "qmm_gemv_argmax_noalloc", "qmm_gemm", "qmm_gemm_swiglu",
           "qmm_quantize_q8_0", "qmm_gemm_q8act", "qmm_gemv_q8act", "qmm_gemv_concat_q8act",
           "qmm_gemv_swiglu_q8act", "qmm_gemv_argmax_q8act", "qmm_repack_bytes", "qmm_repack", "qmm_gemm_repacked", "qmm_gemm_repacked_kernel",
           "qmm_block_norm", "qmm_moe_route", "qmm_moe_swiglu_work_bytes", "qmm_moe_swiglu", "qmm_moe_down_work_bytes",
           "qmm_moe_down", "qmm_kv_pool_bytes", "qmm_rope", "qmm_rope_freqs", "qmm_kv_append",
           "qmm_attention_work_bytes", "qmm_attention", "qmm_gemm_path", "qmm_gemm_q8act_path", "qmm_gemm_kernel", "qmm_gemm_swiglu_kernel", "qmm_read_probe", "qmm_blob_bytes", "qmm_block_elems",
           "qmm_block_bytes", "qmm_strerror")

_lib = None


class QmmError(RuntimeError):
    def __init__(self, code: int, what: str):
        super().__init__(f"{what}: {strerror(code)} (status {code})")
        self.code = code


def lib():
    """The loaded libqmm.so; raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with `python -m gguf_block_quant_qmm_amd.build`")
        L = ctypes.CDLL(LIB_PATH)
        i64, vp, ci = ctypes.c_int64, ctypes.c_void_p, ctypes.c_int
        L.qmm_gemv.argtypes = [vp, ci, i64, i64, vp, vp, vp]
        L.qmm_gemv.restype = ci
        L.qmm_gemv_concat.argtypes = [ci, vp, vp, ci, i64, vp, vp, vp]
        L.qmm_gemv_concat.restype = ci
        L.qmm_gemv_swiglu.argtypes = [vp, vp, ci, i64, i64, vp, vp, vp]
        L.qmm_gemv_swiglu.restype = ci
        L.qmm_gemv_argmax.argtypes = [vp, ci, i64, i64, vp, vp, vp, vp, vp]
        L.qmm_gemv_argmax.restype = ci
        L.qmm_gemv_argmax_noalloc.argtypes = [vp, ci, i64, i64, vp, vp, vp, vp]
        L.qmm_gemv_argmax_noalloc.restype = ci
        L.qmm_gemm_swiglu.argtypes = [vp, vp, ci, i64, i64, i64, vp, vp, vp]
        L.qmm_gemm_swiglu.restype = ci
        L.qmm_gemm.argtypes = [vp, ci, i64, i64, i64, vp, vp, vp]
        L.qmm_gemm.restype = ci
        L.qmm_quantize_q8_0.argtypes = [vp, i64, i64, vp, vp, vp]
        L.qmm_quantize_q8_0.restype = ci
        L.qmm_gemm_q8act.argtypes = [vp, ci, i64, i64, i64, vp, vp, vp, vp]
        L.qmm_gemm_q8act.restype = ci
        L.qmm_gemv_q8act.argtypes = [vp, ci, i64, i64, vp, vp, vp]
        L.qmm_gemv_q8act.restype = ci
        L.qmm_gemv_concat_q8act.argtypes = [ci, vp, vp, ci, i64, vp, vp, vp]
        L.qmm_gemv_concat_q8act.restype = ci
        L.qmm_gemv_swiglu_q8act.argtypes = [vp, vp, ci, i64, i64, vp, vp, vp]
        L.qmm_gemv_swiglu_q8act.restype = ci
        L.qmm_gemv_argmax_q8act.argtypes = [vp, ci, i64, i64, vp, vp, vp, vp, vp]
        L.qmm_gemv_argmax_q8act.restype = ci
        L.qmm_repack_bytes.argtypes = [ci, i64, i64]
        L.qmm_repack_bytes.restype = i64
        L.qmm_repack.argtypes = [vp, ci, i64, i64, vp, vp]
        L.qmm_repack.restype = ci
        L.qmm_gemm_repacked.argtypes = [vp, ci, i64, i64, i64, vp, vp, vp]
        L.qmm_gemm_repacked.restype = ci
        L.qmm_gemm_repacked_kernel.argtypes = [ci, i64, i64, i64]
        L.qmm_gemm_repacked_kernel.restype = ci
        L.qmm_gemm_path.argtypes = [ci, i64, i64, i64]
        L.qmm_gemm_path.restype = ci
        L.qmm_gemm_q8act_path.argtypes = [ci, i64, i64, i64]
        L.qmm_gemm_q8act_path.restype = ci
        L.qmm_gemm_swiglu_kernel.argtypes = [ci, i64, i64, i64]
        L.qmm_gemm_swiglu_kernel.restype = ci
        L.qmm_gemm_kernel.argtypes = [ci, i64, i64, i64]
        L.qmm_gemm_kernel.restype = ci
        L.qmm_read_probe.argtypes = [vp, i64, vp, vp]
        L.qmm_read_probe.restype = ci
        f64 = ctypes.c_double
        L.qmm_block_norm.argtypes = [vp, vp, vp, i64, f64, vp, vp, vp, f64, i64, i64, vp, vp, vp, vp]
        L.qmm_block_norm.restype = ci
        L.qmm_moe_route.argtypes = [vp, vp, i64, i64, ci, i64, i64, ci, i64, ci, f64, vp, vp, vp]
        L.qmm_moe_route.restype = ci
        for f in (L.qmm_moe_swiglu_work_bytes, L.qmm_moe_down_work_bytes):
            f.argtypes = [ci, i64, i64, i64, i64, i64]
            f.restype = i64
        L.qmm_moe_swiglu.argtypes = [vp, vp, ci, i64, i64, i64, i64, i64, vp, vp, vp, vp, i64, vp]
        L.qmm_moe_swiglu.restype = ci
        L.qmm_moe_down.argtypes = [vp, ci, i64, i64, i64, i64, i64, vp, vp, vp, vp, vp, vp, i64, vp]
        L.qmm_moe_down.restype = ci
        L.qmm_kv_pool_bytes.argtypes = [ci, i64, i64, i64, i64]
        L.qmm_kv_pool_bytes.restype = i64
        L.qmm_rope.argtypes = [vp, i64, i64, i64, i64, vp, vp, i64, ci, f64, vp, i64, vp]
        L.qmm_rope.restype = ci
        L.qmm_rope_freqs.argtypes = [i64, f64, f64, f64, f64, f64, vp, vp, vp]
        L.qmm_rope_freqs.restype = ci
        L.qmm_kv_append.argtypes = [vp, vp, vp, i64, vp, i64, vp, i64, ci, f64, vp, vp, vp, f64, vp, i64, i64, vp, vp]
        L.qmm_kv_append.restype = ci
        L.qmm_attention_work_bytes.argtypes = [vp, vp, i64]
        L.qmm_attention_work_bytes.restype = i64
        L.qmm_attention.argtypes = [vp, vp, vp, i64, i64, f64, ci, i64, f64, vp, vp, i64, vp]
        L.qmm_attention.restype = ci
        L.qmm_blob_bytes.argtypes = [ci, i64, i64]
        L.qmm_blob_bytes.restype = i64
        L.qmm_block_elems.argtypes = [ci]
        L.qmm_block_bytes.argtypes = [ci]
        L.qmm_strerror.argtypes = [ci]
        L.qmm_strerror.restype = ctypes.c_char_p
        _lib = L
    return _lib


def strerror(code: int) -> str:
    return lib().qmm_strerror(code).decode()


def block_elems(dtype: int) -> int:
    return lib().qmm_block_elems(dtype)


def block_bytes(dtype: int) -> int:
    return lib().qmm_block_bytes(dtype)


def blob_bytes(dtype: int, M: int, K: int) -> int:
    return lib().qmm_blob_bytes(dtype, M, K)


def gemm_path(dtype: int, M: int, K: int, N: int) -> int:
    return lib().qmm_gemm_path(dtype, M, K, N)


QMM_KERNEL_GEMV, QMM_KERNEL_GEMV_TOKENS = 100, 101


def q8act_kernel(dtype: int, M: int, K: int, N: int) -> int:
    """0: qmm_gemm_q8act runs token groups (single-token bits); 1: the int8 matrix cores."""
    return lib().qmm_gemm_q8act_path(dtype, M, K, N)


def swiglu_kernel(dtype: int, M: int, K: int, N: int) -> int:
    """Form qmm_gemm_swiglu runs for these sizes (see include/qmm.h)."""
    return lib().qmm_gemm_swiglu_kernel(dtype, M, K, N)


def gemm_kernel(dtype: int, M: int, K: int, N: int) -> int:
    """Id of the kernel qmm_gemm runs for these sizes (see include/qmm.h)."""
    return lib().qmm_gemm_kernel(dtype, M, K, N)


def qmm_read_probe(buf, nbytes: int, out, stream=None) -> None:
    """A plain streaming read of nbytes of buf (diagnostic read ceiling)."""
    import torch
    rc = lib().qmm_read_probe(_addr(buf, nbytes, "buf"), nbytes,
                              _addr(out, 4 * QMM_READ_PROBE_OUT_FLOATS, "out", torch.float32), _stream(stream))
    if rc != QMM_OK:
        raise QmmError(rc, "qmm_read_probe")


def tolerance(dtype: int, M: int, K: int, N: int) -> float:
    """Relative tolerance (of sum |w x|) that the chosen path guarantees."""
    return 2e-3 if gemm_path(dtype, M, K, N) == 1 else 1e-5


def _addr(t, nbytes: int | None, what: str, torch_dtype=None) -> int:
    if t is None:
        return 0
    if isinstance(t, int):
        return t
    if not t.is_cuda:
        raise ValueError(f"{what} must be a device tensor")
    if not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous")
    if torch_dtype is not None and t.dtype is not torch_dtype:
        raise ValueError(f"{what} must be {torch_dtype}, got {t.dtype}")
    if nbytes is not None and t.nbytes < nbytes:
        raise ValueError(f"{what} holds {t.nbytes} bytes, needs {nbytes}")
    return t.data_ptr()


def _stream(stream) -> int:
    if stream is None:
        import torch
        # the handle alone: building a Stream object costs 2.6 us, as much as the launch itself
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        if raw is not None:
            return raw(torch.cuda.current_device())
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def qmm_gemv(w, dtype: int, M: int, K: int, x, y, stream=None) -> None:
    import torch
    nb = blob_bytes(dtype, M, K)
    rc = lib().qmm_gemv(_addr(w, nb or None, "w_blob"), dtype, M, K,
                        _addr(x, 4 * K, "x", torch.float32), _addr(y, 4 * M, "y", torch.float32),
                        _stream(stream))
    if rc != QMM_OK:
        raise QmmError(rc, "qmm_gemv")


def qmm_gemm(w, dtype: int, M: int, K: int, N: int, X, Y, stream=None) -> None:
    import torch
    nb = blob_bytes(dtype, M, K)
    rc = lib().qmm_gemm(_addr(w, nb or None, "w_blob"), dtype, M, K, N,
                        _addr(X, 4 * N * K, "X", torch.float32), _addr(Y, 4 * N * M, "Y", torch.float32),
                        _stream(stream))
    if rc != QMM_OK:
        raise QmmError(rc, "qmm_gemm")


def repack_bytes(dtype: int, M: int, K: int) -> int:
    return lib().qmm_repack_bytes(dtype, M, K)


def gemm_repacked_kernel(dtype: int, M: int, K: int, N: int) -> int:
    return lib().qmm_gemm_repacked_kernel(dtype, M, K, N)


def qmm_repack(w, dtype: int, M: int, K: int, packed, stream=None) -> None:
    rc = lib().qmm_repack(_addr(w, blob_bytes(dtype, M, K) or None, "w_blob"), dtype, M, K,
                          _addr(packed, repack_bytes(dtype, M, K) or None, "packed"), _stream(stream))
    if rc != QMM_OK:
        raise QmmError(rc, "qmm_repack")


def qmm_gemm_repacked(packed, dtype: int, M: int, K: int, N: int, X, Y, stream=None) -> None:
    import torch
    rc = lib().qmm_gemm_repacked(_addr(packed, repack_bytes(dtype, M, K) or None, "packed"), dtype, M, K, N,
                                 _addr(X, 4 * N * K, "X", torch.float32), _addr(Y, 4 * N * M, "Y", torch.float32),
                                 _stream(stream))
    if rc != QMM_OK:
        raise QmmError(rc, "qmm_gemm_repacked")


def qmm_gemv_concat(ws, dtype: int, Ms, K: int, x, ys, stream=None) -> None:
    import torch
    n = len(ws)
    if not (len(Ms) == n == len(ys)):
        raise ValueError("ws, Ms and ys need one entry per matrix")
    blobs = (ctypes.c_void_p * max(n, 1))(*[_addr(w, blob_bytes(dtype, M, K) or None, f"ws[{i}]")
                                            for i, (w, M) in enumerate(zip(ws, Ms))])
    rows = (ctypes.c_int64 * max(n, 1))(*[int(M) for M in Ms])
    outs = (ctypes.c_void_p * max(n, 1))(*[_addr(y, 4 * M, f"ys[{i}]", torch.float32)
                                           for i, (y, M) in enumerate(zip(ys, Ms))])
    rc = lib().qmm_gemv_concat(n, blobs, rows, dtype, K, _addr(x, 4 * K, "x", torch.float32), outs,
                               _stream(stream))
    if rc != QMM_OK:
        raise QmmError(rc, "qmm_gemv_concat")


def qmm_gemv_swiglu(gate, up, dtype: int, M: int, K: int, x, out, stream=None) -> None:
    import torch
    nb = blob_bytes(dtype, M, K) or None
    rc = lib().qmm_gemv_swiglu(_addr(gate, nb, "gate"), _addr(up, nb, "up"), dtype, M, K,
                               _addr(x, 4 * K, "x", torch.float32), _addr(out, 4 * M, "out", torch.float32),
                               _stream(stream))
    if rc != QMM_OK:
        raise QmmError(rc, "qmm_gemv_swiglu")


def qmm_gemv_argmax(w, dtype: int, M: int, K: int, x, work, index, value=None, stream=None) -> None:
    import torch
    rc = lib().qmm_gemv_argmax(_addr(w, blob_bytes(dtype, M, K) or None, "w_blob"), dtype, M, K,
                               _addr(x, 4 * K, "x", torch.float32), _addr(work, QMM_ARGMAX_WORK_BYTES, "work"),
                               _addr(index, 8, "index", torch.int64), _addr(value, 4, "value", torch.float32),
                               _stream(stream))
    if rc != QMM_OK:
        raise QmmError(rc, "qmm_gemv_argmax")


def qmm_gemv_argmax_noalloc(w, dtype: int, M: int, K: int, x, index, value=None, stream=None) -> None:
    import torch
    rc = lib().qmm_gemv_argmax_noalloc(_addr(w, blob_bytes(dtype, M, K) or None, "w_blob"), dtype, M, K,
                                       _addr(x, 4 * K, "x", torch.float32), _addr(index, 8, "index", torch.int64),
                                       _addr(value, 4, "value", torch.float32), _stream(stream))
    if rc != QMM_OK:
        raise QmmError(rc, "qmm_gemv_argmax_noalloc")


def qmm_gemm_swiglu(gate, up, dtype: int, M: int, K: int, N: int, X, out, stream=None) -> None:
    import torch
    nb = blob_bytes(dtype, M, K) or None
    rc = lib().qmm_gemm_swiglu(_addr(gate, nb, "gate"), _addr(up, nb, "up"), dtype, M, K, N,
                               _addr(X, 4 * N * K, "X", torch.float32), _addr(out, 4 * N * M, "out", torch.float32),
                               _stream(stream))
    if rc != QMM_OK:
        raise QmmError(rc, "qmm_gemm_swiglu")


def qmm_quantize_q8_0(X, N: int, K: int, scales, quants, stream=None) -> None:
    import torch
    nb = K // 32 if K > 0 else 0
    rc = lib().qmm_quantize_q8_0(_addr(X, 4 * N * K, "X", torch.float32), N, K,
                                 _addr(scales, 4 * N * nb, "scales", torch.float32),
                                 _addr(quants, N * K, "quants", torch.int8), _stream(stream))
    if rc != QMM_OK:
        raise QmmError(rc, "qmm_quantize_q8_0")


def qmm_gemm_q8act(w, dtype: int, M: int, K: int, N: int, scales, quants, Y, stream=None) -> None:
    import torch
    nb = blob_bytes(dtype, M, K)
    rc = lib().qmm_gemm_q8act(_addr(w, nb or None, "w_blob"), dtype, M, K, N,
                              _addr(scales, 4 * N * (K // 32), "scales", torch.float32),
                              _addr(quants, N * K, "quants", torch.int8), _addr(Y, 4 * N * M, "Y", torch.float32),
                              _stream(stream))
    if rc != QMM_OK:
        raise QmmError(rc, "qmm_gemm_q8act")


def qmm_gemv_q8act(w, dtype: int, M: int, K: int, x, y, stream=None) -> None:
    import torch
    nb = blob_bytes(dtype, M, K)
    rc = lib().qmm_gemv_q8act(_addr(w, nb or None, "w_blob"), dtype, M, K,
                              _addr(x, 4 * K, "x", torch.float32), _addr(y, 4 * M, "y", torch.float32),
                              _stream(stream))
    if rc != QMM_OK:
        raise QmmError(rc, "qmm_gemv_q8act")


def qmm_gemv_concat_q8act(ws, dtype: int, Ms, K: int, x, ys, stream=None) -> None:
    import torch
    n = len(ws)
    if not (len(Ms) == n == len(ys)):
        raise ValueError("ws, Ms and ys need one entry per matrix")
    blobs = (ctypes.c_void_p * max(n, 1))(*[_addr(w, blob_bytes(dtype, M, K) or None, f"ws[{i}]")
                                            for i, (w, M) in enumerate(zip(ws, Ms))])
    rows = (ctypes.c_int64 * max(n, 1))(*[int(M) for M in Ms])
    outs = (ctypes.c_void_p * max(n, 1))(*[_addr(y, 4 * M, f"ys[{i}]", torch.float32)
                                           for i, (y, M) in enumerate(zip(ys, Ms))])
    rc = lib().qmm_gemv_concat_q8act(n, blobs, rows, dtype, K, _addr(x, 4 * K, "x", torch.float32), outs,
                                     _stream(stream))
    if rc != QMM_OK:
        raise QmmError(rc, "qmm_gemv_concat_q8act")


def qmm_gemv_swiglu_q8act(gate, up, dtype: int, M: int, K: int, x, out, stream=None) -> None:
    import torch
    nb = blob_bytes(dtype, M, K) or None
    rc = lib().qmm_gemv_swiglu_q8act(_addr(gate, nb, "gate"), _addr(up, nb, "up"), dtype, M, K,
                                     _addr(x, 4 * K, "x", torch.float32), _addr(out, 4 * M, "out", torch.float32),
                                     _stream(stream))
    if rc != QMM_OK:
        raise QmmError(rc, "qmm_gemv_swiglu_q8act")


def qmm_gemv_argmax_q8act(w, dtype: int, M: int, K: int, x, work, index, value=None, stream=None) -> None:
    import torch
    rc = lib().qmm_gemv_argmax_q8act(_addr(w, blob_bytes(dtype, M, K) or None, "w_blob"), dtype, M, K,
                                     _addr(x, 4 * K, "x", torch.float32), _addr(work, QMM_ARGMAX_WORK_BYTES, "work"),
                                     _addr(index, 8, "index", torch.int64), _addr(value, 4, "value", torch.float32),
                                     _stream(stream))
    if rc != QMM_OK:
        raise QmmError(rc, "qmm_gemv_argmax_q8act")


def qmm_block_norm(residual, N: int, K: int, residual_out=None, block=None, w_post=None, gate=None,
                   gate_stride: int = 0, scale: float = 1.0, w_pre=None, eps: float = 1e-5, H=None, scales=None,
                   quants=None, stream=None) -> None:
    import torch
    f32, row, nb = torch.float32, 4 * N * K, (K // 32 if K > 0 else 0)
    rc = lib().qmm_block_norm(_addr(block, row, "block", f32), _addr(w_post, 4 * K, "w_post", f32),
                              _addr(gate, row if gate_stride else 4 * K, "gate", f32), gate_stride, scale,
                              _addr(residual, row, "residual", f32), _addr(residual_out, row, "residual_out", f32),
                              _addr(w_pre, 4 * K, "w_pre", f32), eps, N, K, _addr(H, row, "H", f32),
                              _addr(scales, 4 * N * nb, "scales", f32), _addr(quants, N * K, "quants", torch.int8),
                              _stream(stream))
    if rc != QMM_OK:
        raise QmmError(rc, "qmm_block_norm")


def qmm_moe_route(logits, N: int, E: int, topk: int, ids, weights, bias=None, scoring: int = QMM_ROUTE_SOFTMAX,
                  groups: int = 1, topk_groups: int = 1, group_top: int = 1, renorm: bool = True, scale: float = 1.0,
                  stream=None) -> None:
    import torch
    rc = lib().qmm_moe_route(_addr(logits, 4 * N * E, "logits", torch.float32), _addr(bias, 4 * E, "bias", torch.float32),
                             N, E, scoring, groups, topk_groups, group_top, topk, int(bool(renorm)), scale,
                             _addr(ids, 4 * N * topk, "ids", torch.int32),
                             _addr(weights, 4 * N * topk, "weights", torch.float32), _stream(stream))
    if rc != QMM_OK:
        raise QmmError(rc, "qmm_moe_route")


def moe_swiglu_work_bytes(dtype: int, E: int, M: int, K: int, N: int, T: int) -> int:
    """Bytes of work that qmm_moe_swiglu needs for these sizes (0: none)."""
    return lib().qmm_moe_swiglu_work_bytes(dtype, E, M, K, N, T)


def moe_down_work_bytes(dtype: int, E: int, M: int, K: int, N: int, T: int) -> int:
    """Bytes of work that qmm_moe_down needs for these sizes (0: none)."""
    return lib().qmm_moe_down_work_bytes(dtype, E, M, K, N, T)


def _work(work) -> tuple[int, int]:
    """Address and bytes of a work tensor (None or an empty one: no work)."""
    if work is None:
        return 0, 0
    if isinstance(work, int):
        raise ValueError("work must be a device tensor (an address alone has no size)")
    return _addr(work, None, "work"), work.nbytes


def qmm_moe_swiglu(gate, up, dtype: int, E: int, M: int, K: int, N: int, T: int, ids, X, out, work=None,
                   stream=None) -> None:
    import torch
    nb = E * blob_bytes(dtype, M, K) or None
    rc = lib().qmm_moe_swiglu(_addr(gate, nb, "gate"), _addr(up, nb, "up"), dtype, E, M, K, N, T,
                              _addr(ids, 4 * N * T, "ids", torch.int32), _addr(X, 4 * N * K, "X", torch.float32),
                              _addr(out, 4 * N * T * M, "out", torch.float32), *_work(work), _stream(stream))
    if rc != QMM_OK:
        raise QmmError(rc, "qmm_moe_swiglu")


def qmm_moe_down(w, dtype: int, E: int, M: int, K: int, N: int, T: int, ids, weights, H, Y, residual=None, work=None,
                 stream=None) -> None:
    import torch
    rc = lib().qmm_moe_down(_addr(w, E * blob_bytes(dtype, M, K) or None, "w_blob"), dtype, E, M, K, N, T,
                            _addr(ids, 4 * N * T, "ids", torch.int32),
                            _addr(weights, 4 * N * T, "weights", torch.float32),
                            _addr(H, 4 * N * T * K, "H", torch.float32),
                            _addr(residual, 4 * N * M, "residual", torch.float32),
                            _addr(Y, 4 * N * M, "Y", torch.float32), *_work(work), _stream(stream))
    if rc != QMM_OK:
        raise QmmError(rc, "qmm_moe_down")


def _current_device() -> int:
    import torch
    raw = getattr(torch._C, "_cuda_getDevice", None)  # the index alone: torch.cuda.current_device costs four times as much
    return raw() if raw is not None and torch.cuda.is_initialized() else torch.cuda.current_device()


def _on(dev, t, need: int, what: str, dtype) -> int:
    """Address of a contiguous tensor of at least `need` values on device `dev`,
    the current one (the kernels run there); None: 0; an address as it is."""
    if t is None:
        return 0
    if type(t) is int:
        return t
    if t.get_device() != dev:
        raise ValueError(f"{what} must be a tensor of the current device cuda:{dev}, it is on {t.device}")
    if t.dtype is not dtype:
        raise ValueError(f"{what} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous")
    if t.numel() < need:
        raise ValueError(f"{what} holds {t.numel()} values, needs {need}")
    return t.data_ptr()


def _rows(dev, t, rows: int, width: int, stride: int, what: str, dtype) -> int:
    """Address of f32 rows of `width` values that lie `stride` values apart (0:
    side by side).  The tensor may be a view into wider rows (columns of a fused
    projection, [rows][heads][dim] too), or flat; what the rows reach must lie inside
    its storage."""
    if not stride or t is None or type(t) is int:
        return _on(dev, t, rows * width, what, dtype)
    if t.get_device() != dev:
        raise ValueError(f"{what} must be a tensor of the current device cuda:{dev}, it is on {t.device}")
    if t.dtype is not dtype:
        raise ValueError(f"{what} must be {dtype}, got {t.dtype}")
    if t.dim() == 2 and t.stride() == (stride, 1) and t.shape[0] >= rows and t.shape[1] >= width:
        return t.data_ptr()
    if t.dim() > 1 and t.shape[0] > 0:
        if t.shape[0] > 1 and t.stride(0) != stride or not t[0].is_contiguous():
            raise ValueError(f"{what} must have rows {stride} values apart, each contiguous")
        if (t.shape[0] > 1 or rows == 1) and (t.shape[0] < rows or t[0].numel() < width):
            raise ValueError(f"{what} holds {t.shape[0]} rows of {t[0].numel()} values, needs {rows} of {width}")
    elif t.dim() and t.stride(-1) != 1:
        raise ValueError(f"{what} must have rows {stride} values apart")
    if rows > 0 and width > 0:
        held = t.untyped_storage().nbytes() // 4 - t.storage_offset()
        if held < (rows - 1) * stride + width:
            raise ValueError(f"{what} holds {held} values from its start, needs {(rows - 1) * stride + width}")
    return t.data_ptr()


def _raw_stream(stream, dev: int) -> int:
    if stream is None:
        import torch
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        if raw is not None:
            return raw(dev)
    return _stream(stream)


def kv_pool_bytes(dtype: int, pages: int, page: int, heads: int, dim: int) -> int:
    """Bytes of the key pool, and of the value pool, of a paged cache."""
    return lib().qmm_kv_pool_bytes(dtype, pages, page, heads, dim)


class _KvCacheStruct(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("pages", ctypes.c_int64), ("dtype", ctypes.c_int32),
                ("page", ctypes.c_int32), ("heads", ctypes.c_int32), ("dim", ctypes.c_int32)]


class _KvBatchStruct(ctypes.Structure):
    _fields_ = [("table", ctypes.c_void_p), ("lens", ctypes.c_void_p), ("starts", ctypes.c_void_p),
                ("seqs", ctypes.c_int64), ("max_pages", ctypes.c_int64), ("table_stride", ctypes.c_int64),
                ("max_new", ctypes.c_int64), ("rows", ctypes.c_int64)]


class KvCache:
    """A paged key-value cache: two device pools of kv_pool_bytes(...) bytes
    (any tensor type), described for the calls that take it (qmm_kv_cache)."""

    def __init__(self, k, v, dtype: int, pages: int, page: int, heads: int, dim: int):
        need = kv_pool_bytes(dtype, pages, page, heads, dim)
        if not need:  # before the struct's 32-bit fields cut a size down to a valid one
            raise QmmError(QMM_ERR_SHAPE if dtype in (QMM_F16, QMM_Q8_0) else QMM_ERR_DTYPE, "KvCache")
        self.k, self.v = k, v
        self.dtype, self.pages, self.page, self.heads, self.dim = dtype, pages, page, heads, dim
        self.struct = _KvCacheStruct(_addr(k, need, "k"), _addr(v, need, "v"), pages, dtype, page, heads, dim)
        self.ref = ctypes.addressof(self.struct)
        self.devices = {t.get_device() for t in (k, v) if not isinstance(t, int) and t is not None}

    def _check(self, dev: int) -> None:
        if any(d != dev for d in self.devices):
            raise ValueError(f"the cache's pools must be tensors of the current device cuda:{dev}")


class KvBatch:
    """The sequences of a call and their new tokens (qmm_kv_batch): the page
    table int32 [seqs][table_stride], lens int32 [seqs], starts int32 [seqs + 1] or
    None.  The tensors may change between calls; they are read on the device."""

    def __init__(self, table, lens, seqs: int, max_pages: int, max_new: int, rows: int, starts=None,
                 table_stride: int = 0):
        import torch
        i32 = torch.int32
        for v in (seqs, max_pages, max_new, rows, table_stride):
            if not 0 <= v < 1 << 62:  # a 64-bit field would cut it
                raise QmmError(QMM_ERR_SHAPE, "KvBatch")
        self.table, self.lens, self.starts = table, lens, starts
        self.seqs, self.max_pages, self.max_new, self.rows = seqs, max_pages, max_new, rows
        wide = (seqs - 1) * (table_stride or max_pages) + max_pages
        self.struct = _KvBatchStruct(_addr(table, 4 * wide, "table", i32), _addr(lens, 4 * seqs, "lens", i32),
                                     _addr(starts, 4 * (seqs + 1), "starts", i32), seqs, max_pages, table_stride, max_new,
                                     rows)
        self.ref = ctypes.addressof(self.struct)
        self.devices = {t.get_device() for t in (table, lens, starts) if not isinstance(t, int) and t is not None}

    def _check(self, dev: int) -> None:
        if any(d != dev for d in self.devices):
            raise ValueError(f"the batch's arrays must be tensors of the current device cuda:{dev}")


def qmm_rope_freqs(rot: int, base: float, freqs, factor: float = 1.0, context: float = 0.0, beta_fast: float = 32.0,
                   beta_slow: float = 1.0, factors=None, stream=None) -> None:
    import torch
    dev, f32 = _current_device(), torch.float32
    rc = lib().qmm_rope_freqs(rot, base, factor, context, beta_fast, beta_slow, _on(dev, factors, rot // 2, "factors", f32),
                              _on(dev, freqs, rot // 2, "freqs", f32), _raw_stream(stream, dev))
    if rc != QMM_OK:
        raise QmmError(rc, "qmm_rope_freqs")


def qmm_rope(X, N: int, H: int, D: int, pos, freqs, rot: int, Y, layout: int = QMM_ROPE_HALF, mscale: float = 1.0,
             x_stride: int = 0, y_stride: int = 0, stream=None) -> None:
    import torch
    dev, f32 = _current_device(), torch.float32
    rc = lib().qmm_rope(_rows(dev, X, N, H * D, x_stride, "X", f32), x_stride, N, H, D,
                        _on(dev, pos, N, "pos", torch.int32), _on(dev, freqs, rot // 2, "freqs", f32), rot, layout, mscale,
                        _rows(dev, Y, N, H * D, y_stride, "Y", f32), y_stride, _raw_stream(stream, dev))
    if rc != QMM_OK:
        raise QmmError(rc, "qmm_rope")


def qmm_kv_append(cache: KvCache, batch: KvBatch, K, V, freqs=None, rot: int = 0, layout: int = QMM_ROPE_HALF,
                  mscale: float = 1.0, pos=None, k_norm=None, q_norm=None, eps: float = 1e-5, Q=None, q_heads: int = 0,
                  q_out=None, q_stride: int = 0, k_stride: int = 0, v_stride: int = 0, stream=None) -> None:
    import torch
    dev, f32 = _current_device(), torch.float32
    D, rows = cache.struct.dim, batch.struct.rows  # what the call will use
    cache._check(dev)
    batch._check(dev)
    wide = cache.struct.heads * D
    rc = lib().qmm_kv_append(cache.ref, batch.ref, _rows(dev, K, rows, wide, k_stride, "K", f32), k_stride,
                             _rows(dev, V, rows, wide, v_stride, "V", f32), v_stride,
                             _on(dev, freqs, rot // 2, "freqs", f32), rot, layout, mscale,
                             _on(dev, pos, rows, "pos", torch.int32), _on(dev, k_norm, D, "k_norm", f32),
                             _on(dev, q_norm, D, "q_norm", f32), eps, _rows(dev, Q, rows, q_heads * D, q_stride, "Q", f32),
                             q_stride, q_heads, _on(dev, q_out, rows * q_heads * D, "q_out", f32), _raw_stream(stream, dev))
    if rc != QMM_OK:
        raise QmmError(rc, "qmm_kv_append")


def attention_work_bytes(cache: KvCache, batch: KvBatch, q_heads: int) -> int:
    """Bytes of work that qmm_attention needs for these sizes (0: none)."""
    return lib().qmm_attention_work_bytes(cache.ref, batch.ref, q_heads)


def qmm_attention(cache: KvCache, batch: KvBatch, Q, q_heads: int, out, scale: float | None = None, causal: bool = True,
                  window: int = 0, softcap: float = 0.0, work=None, q_stride: int = 0, stream=None) -> None:
    """scale None: 1 / sqrt(dim)."""
    import torch
    dev, f32 = _current_device(), torch.float32
    D, rows = cache.struct.dim, batch.struct.rows  # what the call will use
    cache._check(dev)
    batch._check(dev)
    if work is not None and not isinstance(work, int) and work.get_device() != dev:
        raise ValueError(f"work must be a tensor of the current device cuda:{dev}, it is on {work.device}")
    rc = lib().qmm_attention(cache.ref, batch.ref, _rows(dev, Q, rows, q_heads * D, q_stride, "Q", f32), q_stride, q_heads,
                             D ** -0.5 if scale is None else scale, int(bool(causal)), window, softcap,
                             _on(dev, out, rows * q_heads * D, "out", f32), *_work(work), _raw_stream(stream, dev))
    if rc != QMM_OK:
        raise QmmError(rc, "qmm_attention")
