// qmm_moe.hip -- the routed experts' products (include/qmm.h, qmm_moe_swiglu
// and qmm_moe_down): every token has T slots, slot (n, t) runs through expert
// e = ids[n][t], and the experts' M x K matrices lie one after the other.
//
// Few tokens: the GEMV's f32 arithmetic (qmm_units.hpp), memory-bound on the
// chosen experts' bytes.  Many tokens: the matrix cores (qmm_moe_gemm.hip).
// Measured, us and fetched TB/s of a launch (profiler's medians, the experts'
// tensors rotating through 1 GiB), 1 token, 2 of 8 experts, gate/up 14336 x 4096 and
// down 4096 x 14336: Q4_0 28.4 (4.7) and 17.3 (3.9), Q4_1 31.8 (4.6) and 20.2 (3.7),
// Q4_K 31.7 (4.2) and 20.6 (3.3), Q5_K 37.3 (4.3) and 25.0 (3.3), Q8_0 44.6 (5.6) and
// 27.7 (4.5), Q6_K 35.2 (5.5) and 22.7 (4.3).  The K-quants' decoding costs more than
// the reads wait: down of 7 tokens, 8 of 64 experts 4096 x 1024 Q5_K, 40-43 us
// (3.1-3.3 TB/s), 30 of them VALU issue; on inputs that the caches hold, 35.  Times of
// two variants beside each other below are from a captured graph over four inputs.
//
// The few-token kernel cuts a row into units of 64 weights, one per lane, as
// the GEMV does, but an expert's rows are often short (K of a few hundred
// weights), so a row takes 16, 32 or 64 lanes and a wavefront 4, 2 or 1 rows at
// once.  Rows longer than 4096 weights are cut into chunks.  An item is a
// (slot, chunk) pair that a workgroup's rows need: the chunks of x for
// gate/up, T times the chunks of the down rows.  A wavefront keeps its item's
// activations in registers for all rows of the workgroup; the partial sums of
// a row meet in LDS and are added in item order, so the down projection's sum
// over a token's experts needs no second pass and no atomics.
#include <algorithm>
#include <cmath>

#include "qmm_device.hpp"
#include "qmm_internal.hpp"
#include "qmm_units.hpp"

namespace qmm {

namespace {

// The last unit of a row with an odd number of 32-weight blocks holds one
// block: what belongs to the next row is dropped.  A block of 18 or 34 bytes
// ends inside a dword that may reach past the blob, where a bounds-checked
// dword load gives 0, so its last two bytes come from a load of their own.
template <int DT> constexpr bool has_tail = DT == QMM_Q4_0 || DT == QMM_Q8_0;
template <int DT>
__device__ __forceinline__ void keep_first_block(uint32_t (&v)[Unit<DT>::NL], uint32_t tail) {
    constexpr int BB = Geo<DT>::BB;
#pragma unroll
    for (int i = 0; i < Unit<DT>::NL; i++) {
        if (4 * i >= BB) v[i] = 0u;
        else if (4 * i + 2 == BB) v[i] = tail;
    }
}

template <int DT> struct UnitAt {  // a unit's byte offsets with the lane's row added
    static __device__ typename Unit<DT>::Off of(int u, uint32_t row) {
        typename Unit<DT>::Off o = Unit<DT>::lane_off(u);
        if constexpr (DT == QMM_Q6_K) { o.a += row; o.c += row; o.s += row; o.d += row; }
        else if constexpr (DT == QMM_Q4_K || DT == QMM_Q5_K) { o.hdr += row; o.qs += row; }
        else o.a += row;
        return o;
    }
};

// The sum over the LPR lanes of a row, in its last lane.
template <int LPR>
__device__ __forceinline__ float row_sum(float v) {
    if constexpr (LPR == 64) return wave_sum_to_lane63(v);
    v += __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), 0xB1, 0xF, 0xF, true));
    v += __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), 0x4E, 0xF, 0xF, true));
    v += __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), 0x141, 0xF, 0xF, true));
    v += __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), 0x140, 0xF, 0xF, true));
    if constexpr (LPR == 32)
        v += __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), 0x142, 0xA, 0xF, false));
    return v;
}

struct MoeGemvArgs {
    const uint8_t *w0, *w1;    // swiglu: gate and up; down: w0
    const int32_t *ids;
    const float *weights, *residual, *x;
    float *out;
    int64_t M, K, row_bytes, mat_bytes;
    int E, T, nb;              // nb: blocks per row
    int U, C;                  // units per row, chunks of 64 units
    int rows, rtiles;          // rows per workgroup, workgroups per matrix
    int phases;                // wavefronts per item
};

// One workgroup: `rows` rows of one slot's expert (SWI), or of every expert of
// one token.  W wavefronts; items round by round when there are more.
// ODD: an odd number of 32-weight blocks per row.  Two wavefronts per SIMD:
// registers for three spill the activations (gate/up of one token, 8 experts of
// 14336 x 4096 Q4_0, 2 each: 31 us with two, 43 with three).
template <int DT, bool SWI, int LPR, bool ODD>
__global__ void __launch_bounds__(512, 2) moe_gemv_kernel(const MoeGemvArgs a) {
    constexpr int RPW = 64 / LPR, NL = Unit<DT>::NL, NM = SWI ? 2 : 1;
    constexpr int D = 3 * NM * NL <= 60 ? 2 : 1;  // row groups in flight behind the current one
    extern __shared__ __attribute__((aligned(16))) floatx4 xs[];
    const int t = (int)threadIdx.x, lane = t & 63, wave = __builtin_amdgcn_readfirstlane(t >> 6);
    const int W = (int)blockDim.x >> 6;
    const int items = SWI ? a.C : a.T * a.C, per_round = W / a.phases;
    const int64_t job = blockIdx.x / a.rtiles;  // slot (SWI) or token
    const int64_t row0 = (int64_t)(blockIdx.x % a.rtiles) * a.rows;
    const int rows = (int)(a.M - row0 < a.rows ? a.M - row0 : a.rows);
    // LDS: the activations of a round's items, then the partial sums [item of
    // the round][matrix][row]
    constexpr int XU = LPR * 17;                // float4 per item (padded units)
    float *part = reinterpret_cast<float *>(xs + per_round * XU);

    const int in_round = wave / a.phases, phase = wave % a.phases;
    const int ul = lane % LPR, rl = lane / LPR;
    const int groups = (rows + RPW - 1) / RPW;
    if constexpr (SWI) {
        const int e = a.ids[job];
        if (e < 0 || e >= a.E) {                // uniform: no expert, zeros
            for (int r = t; r < rows; r += (int)blockDim.x) a.out[job * a.M + row0 + r] = 0.f;
            return;
        }
    }
    for (int i0 = 0; i0 < items; i0 += per_round) {
        const int item = i0 + in_round;
        const int slot = SWI ? 0 : item / a.C, c = SWI ? item : item % a.C;
        const bool have = in_round < per_round && item < items;
        // activations first: loads return in order, and they need no expert id
        constexpr int XR = LPR / 4;             // float4 per lane of an item's activations
        floatx4 xr[XR];
        const int64_t xrow = SWI ? job / a.T : job * a.T + slot;
        const int64_t xleft = a.K - 4096 * (int64_t)c;
        const Rsrc xrs = make_rsrc_uniform(a.x + xrow * a.K + 4096 * (int64_t)c,
                                           have ? (uint32_t)(4 * (xleft < 4096 ? xleft : 4096)) : 0u);
        const bool stage = phase == 0 && in_round < per_round;
        if (stage) {                            // uniform per wavefront
#pragma unroll
            for (int i = 0; i < XR; i++)
                xr[i] = __builtin_bit_cast(floatx4, __builtin_amdgcn_raw_buffer_load_b128(xrs, 16u * lane, 1024u * i, 0));
        }
        const int e = !have ? -1 : a.ids[SWI ? job : job * a.T + slot];
        const bool live = e >= 0 && e < a.E;    // uniform per wavefront
        const int u = 64 * c + ul;
        const bool active = live && u < a.U;
        const bool half = ODD && u == a.U - 1;
        const int64_t at = (live ? (int64_t)e * a.mat_bytes : 0) + row0 * a.row_bytes;
        const uint32_t mis = (uint32_t)(at & 3);
        const uint32_t bytes = live ? (uint32_t)(rows * a.row_bytes) + mis : 0u;
        const Rsrc rs[2] = {make_rsrc_uniform(a.w0 + (at - mis), bytes),
                            make_rsrc_uniform((SWI ? a.w1 : a.w0) + (at - mis), bytes)};
        const typename Unit<DT>::Off off = UnitAt<DT>::of(active ? u : 0, mis + (uint32_t)rl * (uint32_t)a.row_bytes);
        uint32_t buf[D + 1][NM][NL], tail[D + 1][NM];
        auto fetch = [&](int g, uint32_t (&b)[NM][NL], uint32_t (&tl)[NM]) {
            const uint32_t so = (uint32_t)g * (uint32_t)(RPW * a.row_bytes);
#pragma unroll
            for (int m = 0; m < NM; m++) {
                Unit<DT>::load(rs[m], so, off, b[m]);
                if constexpr (ODD && has_tail<DT>)
                    tl[m] = (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(rs[m], off.a + (Geo<DT>::BB & ~3u), so, 0);
                else tl[m] = 0u;
            }
        };
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int s = 0; s < D; s++) fetch(phase + s * a.phases, buf[s], tail[s]);
        if (i0 > 0) __syncthreads();            // the round before is done with xs
        if (stage) {
#pragma unroll
            for (int i = 0; i < XR; i++) xs[in_round * XU + xslot<true>(lane + 64 * i)] = xr[i];
        }
        __syncthreads();
        float xv[64];
        x_from_lds<DT, true>(xs + (in_round < per_round ? in_round : 0) * XU, active ? ul : 0, xv);
        __builtin_amdgcn_sched_barrier(0);
        float wt = 1.f;
        if constexpr (!SWI) wt = live ? a.weights[job * a.T + slot] : 0.f;
        const int mine = in_round < per_round ? groups : 0;
        for (int g0 = phase; g0 < mine; g0 += (D + 1) * a.phases) {
#pragma unroll
            for (int s = 0; s <= D; s++) {
                const int g = g0 + s * a.phases;
                fetch(g + D * a.phases, buf[(s + D) % (D + 1)], tail[(s + D) % (D + 1)]);
                if (g < mine) {                 // uniform per wavefront
                    float v[NM];
#pragma unroll
                    for (int m = 0; m < NM; m++) {
                        if (half) keep_first_block<DT>(buf[s][m], tail[s][m]);
                        const float d = Unit<DT>::dot(buf[s][m], xv, off);
                        v[m] = row_sum<LPR>(active ? d : 0.f);
                    }
                    const int r = g * RPW + rl;
                    if (ul == LPR - 1 && r < rows) {
#pragma unroll
                        for (int m = 0; m < NM; m++) {
                            // gate/up rounds add up in item order; the down sums of a
                            // round's items are weighted here
                            float *p = part + (in_round * NM + m) * a.rows + r;
                            if constexpr (SWI) *p = i0 > 0 ? *p + v[m] : v[m];
                            else if (live) *p = i0 > 0 ? fmaf(wt, v[m], *p) : wt * v[m];
                            else if (i0 == 0) *p = 0.f;
                        }
                    }
                }
            }
        }
    }
    __syncthreads();
    const int sums = items < per_round ? items : per_round;
    for (int r = t; r < rows; r += (int)blockDim.x) {
        if constexpr (SWI) {
            float g = part[r], up = part[a.rows + r];
            for (int i = 1; i < sums; i++) {
                g += part[2 * i * a.rows + r];
                up += part[(2 * i + 1) * a.rows + r];
            }
            a.out[job * a.M + row0 + r] = silu(g) * up;
        } else {
            float y = part[r];
            for (int i = 1; i < sums; i++) y += part[i * a.rows + r];
            const int64_t o = job * a.M + row0 + r;
            a.out[o] = a.residual ? a.residual[o] + y : y;
        }
    }
}

template <int DT, bool SWI, bool ODD>
void launch_lpr(int lpr, dim3 grid, dim3 block, size_t lds, hipStream_t st, const MoeGemvArgs &a) {
    switch (lpr) {
    case 16: hipLaunchKernelGGL((moe_gemv_kernel<DT, SWI, 16, ODD>), grid, block, lds, st, a); break;
    case 32: hipLaunchKernelGGL((moe_gemv_kernel<DT, SWI, 32, ODD>), grid, block, lds, st, a); break;
    default: hipLaunchKernelGGL((moe_gemv_kernel<DT, SWI, 64, ODD>), grid, block, lds, st, a); break;
    }
}

template <int DT, bool SWI>
hipError_t run_gemv(const void *w0, const void *w1, int64_t E, int64_t M, int64_t K, int64_t N, int64_t T, const int32_t *ids,
                    const float *weights, const float *x, const float *residual, float *out, hipStream_t st, int cus) {
    MoeGemvArgs a;
    a.w0 = static_cast<const uint8_t *>(w0);
    a.w1 = static_cast<const uint8_t *>(w1);
    a.ids = ids;
    a.weights = weights;
    a.residual = residual;
    a.x = x;
    a.out = out;
    a.M = M;
    a.K = K;
    a.nb = (int)(K / Geo<DT>::BS);
    a.row_bytes = (int64_t)a.nb * Geo<DT>::BB;
    a.mat_bytes = M * a.row_bytes;
    a.E = (int)E;
    a.T = (int)T;
    a.U = (int)((K + 63) / 64);
    a.C = (a.U + 63) / 64;
    const int lpr = a.U <= 16 ? 16 : (a.U <= 32 ? 32 : 64);
    const int items = SWI ? a.C : (int)T * a.C;
    // up to 8 wavefronts; several per item when there are few items
    const int per_round = std::min(items, 8);
    a.phases = items == 1 ? 4 : std::max(1, 8 / per_round);
    const int W = per_round * a.phases, rpw = 64 / lpr;
    const int64_t jobs = SWI ? N * T : N;
    // rows per workgroup: 8 wavefronts per CU, as many as run at a time, so that
    // each stages its activations once; whole row groups for every phase.  Against
    // 16 per CU: gate/up of one token, 2 experts of 14336 x 4096 Q4_0, 30.7 against
    // 33.4 us; 8 of 1024 x 2048 Q4_K, 8.7 against 9.8
    const int64_t wgs = std::max<int64_t>(1, (int64_t)cus * 8 / W);
    const int64_t step = (int64_t)rpw * a.phases;
    const int64_t tiles_max = std::max<int64_t>(1, wgs / jobs);  // no last, nearly empty round of workgroups
    int64_t rows = (M + tiles_max - 1) / tiles_max;
    rows = std::max(step, (rows + step - 1) / step * step);
    rows = std::min<int64_t>(rows, std::max<int64_t>(step, 256 / step * step));
    a.rows = (int)rows;
    const int64_t rtiles = (M + rows - 1) / rows;
    a.rtiles = (int)rtiles;
    const size_t lds = (size_t)per_round * ((size_t)lpr * 272 + (SWI ? 2 : 1) * 4 * (size_t)rows);
    const dim3 grid((unsigned)(jobs * rtiles)), block(64 * W);
    if (Geo<DT>::BS == 32 && (a.nb & 1)) launch_lpr<DT, SWI, Geo<DT>::BS == 32>(lpr, grid, block, lds, st, a);
    else launch_lpr<DT, SWI, false>(lpr, grid, block, lds, st, a);
    return hipGetLastError();
}

// Which form, by what the two take.  The few-token kernel spends every slot's
// expert again: its bytes at r1, rows counted as the lanes they occupy (a row of 4
// units takes 16 lanes), and 5 ns for its workgroups.  The matrix cores take 20 us
// for their launches and every touched expert's bytes once, at r2; of E experts S
// slots touch about E (1 - e^(-S/E)).  The rates are those measured while either
// form is slower than its launches (TB/s; caches serve an expert's second slot, so
// r1 can pass the memory's rate).  Few tokens against matrix cores, measured:
//   64 experts, 8 each, gate/up 1024 x 2048, 16 and 24 tokens: Q4_0 48 / 60 us and
//   72 / 62, Q4_1 55 / 61 and 76 / 62, Q4_K 61 / 53 and 89 / 55, Q5_K 74 / 64 and 106 /
//   66, Q8_0 71 / 76 and 102 / 78, Q6_K 68 / 80 and 102 / 81; down 2048 x 1024: Q4_0
//   28 / 38 and 40 / 39, Q4_1 28 / 37 and 43 / 39, Q4_K 31 / 34 and 47 / 34, Q5_K 40 /
//   42 and 61 / 43, Q8_0 35 / 48 and 51 / 49, Q6_K 36 / 49 and 55 / 51
//   8 experts, 2 each, gate/up 14336 x 4096, 4, 8 and 12 tokens: Q4_0 95 / 142, 173 /
//   185, 240 / 198; Q4_1 104 / 143, 201 / 187, 289 / 197; Q4_K 110 / 127, 208 / 175,
//   299 / 188; Q5_K 138 / 156, 263 / 213, 386 / 229; Q8_0 136 / 192, 275 / 247, 415 /
//   263; Q6_K 133 / 198, 262 / 260 (253 / 257 another time), 381 / 272
//   16 experts, 4 each, gate/up 256 x 256 Q4_K, 1024 tokens: 177 / 21
// The rule takes the faster one at all of these points but one (down of 24 tokens in
// Q4_1, 43 against 39).  It counts every slot as live and knows nothing of shared K.
// A measurement build takes QMM_MOE_GEMM_FROM_N = n to decide by the tokens alone.
bool use_gemm(int dtype, int64_t E, int64_t M, int64_t K, int64_t N, int64_t T, bool down) {
    static const int lever = tuning_lever("QMM_MOE_GEMM_FROM_N", 0);
    if (lever) return N >= lever;
    if (N * T > (int64_t(1) << 30) / M) return true;  // the few-token kernel's grid
    struct Rate { int bs, bb; double r1, r2; };
    const Rate f = dtype == QMM_Q4_0   ? Rate{32, 18, 6.0, 2.8}
                   : dtype == QMM_Q4_1 ? Rate{32, 20, 6.0, 3.0}
                   : dtype == QMM_Q8_0 ? Rate{32, 34, 7.5, 3.8}
                   : dtype == QMM_Q4_K ? Rate{256, 144, 5.0, 3.5}
                   : dtype == QMM_Q5_K ? Rate{256, 176, 5.0, 3.4}
                                       : Rate{256, 210, 6.0, 3.0};
    const int64_t U = (K + 63) / 64, lanes = U <= 16 ? 16 : U <= 32 ? 32 : (U + 63) / 64 * 64;
    const double S = (double)(N * T), rows = (down ? 1.0 : 2.0) * (double)M, per = (double)f.bb / f.bs * 1e-6;  // MB a weight
    const double few = S * (rows * 64.0 * (double)lanes * per / f.r1 + 0.005);
    const double many = 20.0 + (double)E * (1.0 - std::exp(-S / (double)E)) * rows * (double)K * per / f.r2;
    return few > many;
}

}  // namespace

int64_t moe_swiglu_work_bytes(int dtype, int64_t E, int64_t M, int64_t K, int64_t N, int64_t T) {
    return use_gemm(dtype, E, M, K, N, T, false) ? moe_gemm_work_bytes(dtype, E, M, K, N, T, false) : 0;
}
int64_t moe_down_work_bytes(int dtype, int64_t E, int64_t M, int64_t K, int64_t N, int64_t T) {
    return use_gemm(dtype, E, M, K, N, T, true) ? moe_gemm_work_bytes(dtype, E, M, K, N, T, true) : 0;
}

hipError_t launch_moe_swiglu(const void *gate, const void *up, int dtype, int64_t E, int64_t M, int64_t K, int64_t N,
                             int64_t T, const int32_t *ids, const float *X, float *out, void *work, hipStream_t st,
                             int cus) {
    if (use_gemm(dtype, E, M, K, N, T, false)) return launch_moe_gemm_swiglu(gate, up, dtype, E, M, K, N, T, ids, X, out, work, st);
#define QMM_CALL(DT) return run_gemv<DT, true>(gate, up, E, M, K, N, T, ids, nullptr, X, nullptr, out, st, cus)
    QMM_MOE_DT(dtype, QMM_CALL)
#undef QMM_CALL
    return hipErrorInvalidValue;
}

hipError_t launch_moe_down(const void *w, int dtype, int64_t E, int64_t M, int64_t K, int64_t N, int64_t T,
                           const int32_t *ids, const float *weights, const float *H, const float *residual, float *Y,
                           void *work, hipStream_t st, int cus) {
    if (use_gemm(dtype, E, M, K, N, T, true)) return launch_moe_gemm_down(w, dtype, E, M, K, N, T, ids, weights, H, residual, Y, work, st);
#define QMM_CALL(DT) return run_gemv<DT, false>(w, nullptr, E, M, K, N, T, ids, weights, H, residual, Y, st, cus)
    QMM_MOE_DT(dtype, QMM_CALL)
#undef QMM_CALL
    return hipErrorInvalidValue;
}

}  // namespace qmm
