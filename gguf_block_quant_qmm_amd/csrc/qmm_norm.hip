// qmm_norm.hip -- the norms after and before a block, fused with the block's
// gate and residual scale (include/qmm.h, qmm_block_norm):
//     p = w_post ? block / sqrt(mean(block^2) + eps) * w_post : block
//     r = residual + scale * gate * p                          (stored, f32)
//     h = r / sqrt(mean(r^2) + eps) * w_pre                    (f32 and/or Q8_0)
//
// The arithmetic is f64 throughout and every stored value is rounded to f32
// once: the f64 FMA rate of gfx950 equals its unpacked f32 rate, a row needs
// ~10 operations per element against 12 or more bytes of memory traffic, and
// the Q8_0 codes of h then do not hang on the order of the sums (a code next
// to a rounding border would).  The squares of f32 values neither overflow nor
// vanish in f64.  h is computed from the rounded r, the value that
// residual_out holds and the next block adds to.
//
// Memory-bound: 4096 rows of 4096 (block, residual in; r, h out) take 51 us, 5.3
// TB/s, the rate of a large copy on this card (5.1).  One read of the inputs and
// one write of the outputs: a row of up to 16384 values lives in registers (a
// wavefront per row up to 1024 values, else a workgroup), the two sums of squares
// are wavefront reductions with DPP moves joined over the workgroup through LDS in
// wavefront order.  Longer rows are read again for each pass, mostly from the
// caches (512 rows of 20480: 38 us, 169 MB fetched for 84 MB of inputs).  One row of
// 4096 is bound by latency: load, two sums, store, 3.1 us (4 to 5 us with a norm
// after the block, between other launches).  These are the profiler's medians over
// inputs that rotate through up to 1 GiB; times of two variants beside each other
// below are from a captured graph over four inputs.
#include "qmm_device.hpp"
#include "qmm_internal.hpp"
#include "qmm_units.hpp"

namespace qmm {

namespace {

template <int CTRL, int ROW_MASK, bool BOUND>
__device__ __forceinline__ double dpp_d(double v) {
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)b, CTRL, ROW_MASK, 0xF, BOUND);
    const uint32_t hi = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)(b >> 32), CTRL, ROW_MASK, 0xF, BOUND);
    return __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
}

// The sum over the wavefront's 64 lanes in a fixed order, in every lane.
__device__ __forceinline__ double wave_sum_f64(double v) {
    v += dpp_d<0xB1, 0xF, true>(v);    // quad_perm 1,0,3,2
    v += dpp_d<0x4E, 0xF, true>(v);    // quad_perm 2,3,0,1
    v += dpp_d<0x141, 0xF, true>(v);   // row_half_mirror
    v += dpp_d<0x140, 0xF, true>(v);   // row_mirror
    v += dpp_d<0x142, 0xA, false>(v);  // row_bcast15
    v += dpp_d<0x143, 0xC, false>(v);  // row_bcast31: the sum, in lane 63
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = __builtin_amdgcn_readlane((int)(uint32_t)b, 63);
    const uint32_t hi = __builtin_amdgcn_readlane((int)(uint32_t)(b >> 32), 63);
    return __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
}

// The same over the workgroup's `waves` wavefronts (uniform; 1 needs no LDS).
__device__ __forceinline__ double group_sum_f64(double v, double *red, int wave, int waves) {
    v = wave_sum_f64(v);
    if (waves == 1) return v;
    if ((threadIdx.x & 63) == 0) red[wave] = v;
    __syncthreads();
    double s = red[0];
    for (int w = 1; w < waves; w++) s += red[w];
    return s;
}

struct NormArgs {
    const float *block, *w_post, *gate, *residual, *w_pre;
    float *r_out, *H, *scales;
    int8_t *quants;
    int64_t N, gate_stride;
    int K;
    double scale, eps;
};

// V consecutive values per load (4: K % 4 == 0; 1: any K).
template <int V> struct Vec;
template <> struct Vec<4> {
    typedef floatx4 T;
    __device__ static T load(Rsrc rs, uint32_t off) { return __builtin_bit_cast(T, __builtin_amdgcn_raw_buffer_load_b128(rs, off, 0, 0)); }
    __device__ static void store(Rsrc rs, uint32_t off, T v) { __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4_t, v), rs, off, 0, 0); }
    __device__ static float get(const T &v, int i) { return v[i]; }
    __device__ static void set(T &v, int i, float f) { v[i] = f; }
};
template <> struct Vec<1> {
    typedef float T;
    __device__ static T load(Rsrc rs, uint32_t off) { return __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(rs, off, 0, 0)); }
    __device__ static void store(Rsrc rs, uint32_t off, T v) { __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(uint32_t, v), rs, off, 0, 0); }
    __device__ static float get(const T &v, int) { return v; }
    __device__ static void set(T &v, int, float f) { v = f; }
};

// Q8_0 codes of four values of h per lane, eight lanes a block: the bits of
// qmm_quantize_q8_0.  Every lane of the wavefront calls it; `in` marks lanes
// inside the row (whole groups of eight, K % 32 == 0).
__device__ __forceinline__ void put_q8(const NormArgs &a, int64_t row, int k, bool in, const floatx4 &h) {
    float d;
    const uint32_t packed = q8_quant4(h, &d);
    if (in) {
        *reinterpret_cast<uint32_t *>(a.quants + row * a.K + k) = packed;
        if ((k & 31) == 0) a.scales[row * (a.K / 32) + k / 32] = (float)(_Float16)d;
    }
}

// A row in registers: NV vectors of V values per thread, the threads of one
// wavefront (WAVE: blockDim.x / 64 rows per workgroup) or of the workgroup.
// Reads past the row's K values give zeros and writes there are dropped
// (bounds-checked buffer accesses), so no access has a branch around it.
template <int V, int NV, bool WAVE>
__global__ void __launch_bounds__(1024) norm_kernel(const NormArgs a) {
    typedef typename Vec<V>::T T;
    __shared__ double red[2][16];
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int waves = WAVE ? 1 : (int)blockDim.x >> 6;
    const int64_t row = WAVE ? (int64_t)blockIdx.x * (blockDim.x >> 6) + wave : (int64_t)blockIdx.x;
    if (WAVE && row >= a.N) return;  // whole wavefronts; no barrier follows in this form
    const int t = WAVE ? (int)threadIdx.x & 63 : (int)threadIdx.x, step = WAVE ? 64 : (int)blockDim.x;
    const uint32_t bytes = 4u * (uint32_t)a.K;
    const bool has_b = a.block != nullptr, has_w = a.w_post != nullptr, has_g = a.gate != nullptr,
               has_n = a.w_pre != nullptr;
    // an absent vector is a resource of no bytes: its loads give zeros and touch nothing
    const Rsrc rres = make_rsrc_uniform(a.residual + row * a.K, bytes);
    const Rsrc rblk = make_rsrc_uniform(has_b ? a.block + row * a.K : a.residual, has_b ? bytes : 0u);
    const Rsrc rwp = make_rsrc_uniform(has_w ? a.w_post : a.residual, has_w ? bytes : 0u);
    const Rsrc rg = make_rsrc_uniform(has_g ? a.gate + row * a.gate_stride : a.residual, has_g ? bytes : 0u);
    const Rsrc rwn = make_rsrc_uniform(has_n ? a.w_pre : a.residual, has_n ? bytes : 0u);
    uint32_t off[NV];
    T blk[NV], res[NV], wp[NV], g[NV], wn[NV];
#pragma unroll
    for (int i = 0; i < NV; i++) off[i] = 4u * V * (uint32_t)(t + i * step);
#pragma unroll
    for (int i = 0; i < NV; i++) blk[i] = Vec<V>::load(rblk, off[i]);
#pragma unroll
    for (int i = 0; i < NV; i++) res[i] = Vec<V>::load(rres, off[i]);
#pragma unroll
    for (int i = 0; i < NV; i++) wp[i] = Vec<V>::load(rwp, off[i]);
#pragma unroll
    for (int i = 0; i < NV; i++) g[i] = Vec<V>::load(rg, off[i]);
#pragma unroll
    for (int i = 0; i < NV; i++) wn[i] = Vec<V>::load(rwn, off[i]);

    double inv = 1.0;
    if (has_w) {  // uniform
        double ss = 0.0;
#pragma unroll
        for (int i = 0; i < NV; i++)
#pragma unroll
            for (int j = 0; j < V; j++) {
                const double v = Vec<V>::get(blk[i], j);
                ss = fma(v, v, ss);
            }
        inv = 1.0 / sqrt(group_sum_f64(ss, red[0], wave, waves) / a.K + a.eps);
    }
    double ss = 0.0;
#pragma unroll
    for (int i = 0; i < NV; i++)
#pragma unroll
        for (int j = 0; j < V; j++) {
            float rv = Vec<V>::get(res[i], j);
            if (has_b) {
                // the scale last: scale / norm alone may be beyond f64
                double p = inv * Vec<V>::get(blk[i], j);
                if (has_w) p *= Vec<V>::get(wp[i], j);
                if (has_g) p *= Vec<V>::get(g[i], j);
                rv = (float)fma(a.scale, p, (double)rv);
            }
            Vec<V>::set(res[i], j, rv);
            ss = fma((double)rv, (double)rv, ss);
        }
    if (a.r_out) {
        const Rsrc ro = make_rsrc_uniform(a.r_out + row * a.K, bytes);
#pragma unroll
        for (int i = 0; i < NV; i++) Vec<V>::store(ro, off[i], res[i]);
    }
    if (!a.H && !a.quants) return;
    inv = 1.0 / sqrt(group_sum_f64(ss, red[1], wave, waves) / a.K + a.eps);
#pragma unroll
    for (int i = 0; i < NV; i++)
#pragma unroll
        for (int j = 0; j < V; j++) {
            double h = inv * Vec<V>::get(res[i], j);
            if (has_n) h *= Vec<V>::get(wn[i], j);
            Vec<V>::set(res[i], j, (float)h);
        }
    if (a.H) {
        const Rsrc ro = make_rsrc_uniform(a.H + row * a.K, bytes);
#pragma unroll
        for (int i = 0; i < NV; i++) Vec<V>::store(ro, off[i], res[i]);
    }
    if constexpr (V == 4) {
        if (a.quants) {
#pragma unroll
            for (int i = 0; i < NV; i++) put_q8(a, row, (int)(off[i] / 4u), off[i] < bytes, res[i]);
        }
    }
}

// Rows longer than the registers hold (K > 16384): one workgroup per row,
// three passes; a thread reads and writes the same elements in each, so
// residual_out may be the residual itself.
template <int V>
__global__ void __launch_bounds__(1024) norm_long_kernel(const NormArgs a) {
    typedef typename Vec<V>::T T;
    __shared__ double red[2][16];
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6), waves = (int)blockDim.x >> 6;
    const int64_t row = blockIdx.x;
    const int nv = a.K / V, t = (int)threadIdx.x, T0 = (int)blockDim.x;
    const T *blk = reinterpret_cast<const T *>(a.block ? a.block + row * a.K : nullptr);
    const T *res = reinterpret_cast<const T *>(a.residual + row * a.K);
    const T *gate = reinterpret_cast<const T *>(a.gate ? a.gate + row * a.gate_stride : nullptr);
    const T *wp = reinterpret_cast<const T *>(a.w_post), *wn = reinterpret_cast<const T *>(a.w_pre);
    T *ro = reinterpret_cast<T *>(a.r_out ? a.r_out + row * a.K : nullptr);
    T *H = reinterpret_cast<T *>(a.H ? a.H + row * a.K : nullptr);
    double inv = 1.0, ss = 0.0;
    if (wp && blk) {
        for (int i = t; i < nv; i += T0) {
            const T b = blk[i];
#pragma unroll
            for (int j = 0; j < V; j++) {
                const double v = Vec<V>::get(b, j);
                ss = fma(v, v, ss);
            }
        }
        inv = 1.0 / sqrt(group_sum_f64(ss, red[0], wave, waves) / a.K + a.eps);
    }
    ss = 0.0;
    for (int i = t; i < nv; i += T0) {
        T r = res[i];
        if (blk) {
            const T b = blk[i];
#pragma unroll
            for (int j = 0; j < V; j++) {
                double p = inv * Vec<V>::get(b, j);
                if (wp) p *= Vec<V>::get(wp[i], j);
                if (gate) p *= Vec<V>::get(gate[i], j);
                Vec<V>::set(r, j, (float)fma(a.scale, p, (double)Vec<V>::get(r, j)));
            }
        }
        if (ro) ro[i] = r;
#pragma unroll
        for (int j = 0; j < V; j++) ss = fma((double)Vec<V>::get(r, j), (double)Vec<V>::get(r, j), ss);
    }
    if (!H && !a.quants) return;
    inv = 1.0 / sqrt(group_sum_f64(ss, red[1], wave, waves) / a.K + a.eps);
    const T *rr = ro ? ro : res;
    const int rounds = (nv + T0 - 1) / T0;  // uniform: the quantizer needs whole wavefronts
    for (int k = 0; k < rounds; k++) {
        const int i = t + k * T0;
        const bool in = i < nv;
        T h{};
        if (in) {
            const T r = rr[i];
#pragma unroll
            for (int j = 0; j < V; j++) {
                double v = inv * Vec<V>::get(r, j);
                if (wn) v *= Vec<V>::get(wn[i], j);
                Vec<V>::set(h, j, (float)v);
            }
            if (H) H[i] = h;
        }
        if constexpr (V == 4) {
            if (a.quants) put_q8(a, row, 4 * i, in, h);
        }
    }
}

template <int V>
hipError_t launch_v(const NormArgs &a, hipStream_t st) {
    const int64_t nv = (a.K + V - 1) / V;  // vectors per row
    if (nv <= 256) {
        // a wavefront per row, four rows per workgroup
        const unsigned wpb = a.N >= 4 ? 4 : (unsigned)a.N;
        const dim3 grid((unsigned)((a.N + wpb - 1) / wpb)), block(64 * wpb);
        if (nv <= 64) hipLaunchKernelGGL((norm_kernel<V, 1, true>), grid, block, 0, st, a);
        else if (nv <= 128) hipLaunchKernelGGL((norm_kernel<V, 2, true>), grid, block, 0, st, a);
        else hipLaunchKernelGGL((norm_kernel<V, 4, true>), grid, block, 0, st, a);
    } else if (nv <= (V == 4 ? 4096 : 16384)) {
        // few wavefronts with many loads each.  4096 x 4096: 256 threads a row
        // (4 vectors each) 52 us, 512 54, 1024 67.5, 128 92; one row: 3.9, 4.6, 4.8,
        // 7.1 us.  Odd widths: 37 x 4099 with 8 values a thread 5.2 us, 16 5.6
        const int64_t per = V == 4 ? (nv <= 512 ? 2 : 4) : (nv <= 1024 ? 4 : nv <= 4608 ? 8 : 16);
        const dim3 grid((unsigned)a.N), block((unsigned)(((nv + per - 1) / per + 63) / 64 * 64));
        switch (per) {
        case 2: if constexpr (V == 4) hipLaunchKernelGGL((norm_kernel<V, 2, false>), grid, block, 0, st, a); break;
        case 4: hipLaunchKernelGGL((norm_kernel<V, 4, false>), grid, block, 0, st, a); break;
        case 8: if constexpr (V == 1) hipLaunchKernelGGL((norm_kernel<V, 8, false>), grid, block, 0, st, a); break;
        default: if constexpr (V == 1) hipLaunchKernelGGL((norm_kernel<V, 16, false>), grid, block, 0, st, a); break;
        }
    } else {
        hipLaunchKernelGGL((norm_long_kernel<V>), dim3((unsigned)a.N), dim3(1024), 0, st, a);
    }
    return hipGetLastError();
}

}  // namespace

hipError_t launch_block_norm(const float *block, const float *w_post, const float *gate, int64_t gate_stride,
                             double scale, const float *residual, float *residual_out, const float *w_pre, double eps,
                             int64_t N, int64_t K, float *H, float *scales, int8_t *quants, hipStream_t st) {
    // a grid holds fewer than 2^32 threads: at most 2^21 rows of 1024 per launch
    constexpr int64_t kRows = int64_t(1) << 21;
    for (int64_t n0 = 0; n0 < N; n0 += kRows) {
        NormArgs a;
        a.block = block ? block + n0 * K : nullptr;
        a.w_post = block ? w_post : nullptr;
        a.gate = block && gate ? gate + n0 * gate_stride : nullptr;
        a.residual = residual + n0 * K;
        a.w_pre = w_pre;
        a.r_out = residual_out ? residual_out + n0 * K : nullptr;
        a.H = H ? H + n0 * K : nullptr;
        a.scales = scales ? scales + n0 * (K / 32) : nullptr;
        a.quants = quants ? quants + n0 * K : nullptr;
        a.N = N - n0 < kRows ? N - n0 : kRows;
        a.gate_stride = gate_stride;
        a.K = (int)K;
        a.scale = scale;
        a.eps = eps;
        const hipError_t e = K % 4 == 0 ? launch_v<4>(a, st) : launch_v<1>(a, st);
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace qmm
