// qmm_moe.hip -- the routed experts' products (include/qmm.h, qmm_moe_swiglu
// and qmm_moe_down): every token has T slots, slot (n, t) runs through expert
// e = ids[n][t], and the experts' M x K matrices lie one after the other.
#include "qmm_device.hpp"
#include "qmm_internal.hpp"
#include "qmm_units.hpp"

namespace qmm {

namespace {

// One row of one expert against one activation row, a wavefront, any layout.
template <int DT>
__device__ __forceinline__ float row_dot(const uint8_t *row, const float *x, int64_t nb, int lane) {
    float acc = 0.f;
    for (int64_t b = lane; b < nb; b += 64) acc += block_dot_generic<DT>(row + b * Geo<DT>::BB, x + b * Geo<DT>::BS);
    return wave_sum(acc);
}

template <int DT>
__global__ void __launch_bounds__(256) moe_swiglu_rows_kernel(const uint8_t *gate, const uint8_t *up, int E, int64_t M,
                                                              int64_t K, int64_t slots, int T, const int32_t *ids,
                                                              const float *X, float *out) {
    const int lane = (int)threadIdx.x & 63;
    const int64_t nb = K / Geo<DT>::BS, row_bytes = nb * Geo<DT>::BB;
    for (int64_t w = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); w < slots * M; w += (int64_t)gridDim.x * 4) {
        const int64_t slot = w / M, m = w % M;
        const int e = ids[slot];
        float v = 0.f;
        if (e >= 0 && e < E) {
            const int64_t at = ((int64_t)e * M + m) * row_bytes;
            const float *x = X + slot / T * K;
            v = silu(row_dot<DT>(gate + at, x, nb, lane)) * row_dot<DT>(up + at, x, nb, lane);
        }
        if (lane == 0) out[w] = v;
    }
}

template <int DT>
__global__ void __launch_bounds__(256) moe_down_rows_kernel(const uint8_t *w_blob, int E, int64_t M, int64_t K,
                                                            int64_t N, int T, const int32_t *ids, const float *weights,
                                                            const float *H, const float *residual, float *Y) {
    const int lane = (int)threadIdx.x & 63;
    const int64_t nb = K / Geo<DT>::BS, row_bytes = nb * Geo<DT>::BB;
    for (int64_t w = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); w < N * M; w += (int64_t)gridDim.x * 4) {
        const int64_t n = w / M, m = w % M;
        float y = residual ? residual[w] : 0.f;
        for (int t = 0; t < T; t++) {
            const int e = ids[n * T + t];
            if (e < 0 || e >= E) continue;
            const uint8_t *row = w_blob + ((int64_t)e * M + m) * row_bytes;
            y = fmaf(weights[n * T + t], row_dot<DT>(row, H + (n * T + t) * K, nb, lane), y);
        }
        if (lane == 0) Y[w] = y;
    }
}

unsigned rows_grid(int64_t rows) {
    const int64_t g = (rows + 3) / 4;
    return (unsigned)(g < (1 << 20) ? g : (1 << 20));
}

}  // namespace

// Few tokens: a wavefront per row.  A tuning lever of measurement builds only.
static bool use_gemm(int64_t E, int64_t M, int64_t K, int64_t N, int64_t T) {
    static const int lever = tuning_lever("QMM_MOE_GEMM_FROM_N", 8);
    (void)E;
    (void)T;
    return moe_gemm_ok(M, K) && N >= lever;
}

int64_t moe_swiglu_work_bytes(int dtype, int64_t E, int64_t M, int64_t K, int64_t N, int64_t T) {
    return use_gemm(E, M, K, N, T) ? moe_gemm_work_bytes(dtype, E, M, K, N, T, false) : 0;
}
int64_t moe_down_work_bytes(int dtype, int64_t E, int64_t M, int64_t K, int64_t N, int64_t T) {
    return use_gemm(E, M, K, N, T) ? moe_gemm_work_bytes(dtype, E, M, K, N, T, true) : 0;
}

hipError_t launch_moe_swiglu(const void *gate, const void *up, int dtype, int64_t E, int64_t M, int64_t K, int64_t N,
                             int64_t T, const int32_t *ids, const float *X, float *out, void *work, hipStream_t st,
                             int) {
    if (use_gemm(E, M, K, N, T)) return launch_moe_gemm_swiglu(gate, up, dtype, E, M, K, N, T, ids, X, out, work, st);
#define QMM_CALL(DT)                                                                                                   \
    hipLaunchKernelGGL((moe_swiglu_rows_kernel<DT>), dim3(rows_grid(N *T *M)), dim3(256), 0, st, (const uint8_t *)gate, \
                       (const uint8_t *)up, (int)E, M, K, N *T, (int)T, ids, X, out)
    QMM_MOE_DT(dtype, QMM_CALL)
#undef QMM_CALL
    return hipGetLastError();
}

hipError_t launch_moe_down(const void *w, int dtype, int64_t E, int64_t M, int64_t K, int64_t N, int64_t T,
                           const int32_t *ids, const float *weights, const float *H, const float *residual, float *Y,
                           void *work, hipStream_t st, int) {
    if (use_gemm(E, M, K, N, T))
        return launch_moe_gemm_down(w, dtype, E, M, K, N, T, ids, weights, H, residual, Y, work, st);
#define QMM_CALL(DT)                                                                                                  \
    hipLaunchKernelGGL((moe_down_rows_kernel<DT>), dim3(rows_grid(N *M)), dim3(256), 0, st, (const uint8_t *)w, (int)E, \
                       M, K, N, (int)T, ids, weights, H, residual, Y)
    QMM_MOE_DT(dtype, QMM_CALL)
#undef QMM_CALL
    return hipGetLastError();
}

}  // namespace qmm
