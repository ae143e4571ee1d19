// qmm_route.hip -- routing of tokens to experts (include/qmm.h, qmm_moe_route):
//     s = softmax(l) or sigmoid(l);  c = s + bias
//     the topk_groups groups with the largest group scores stay open (a
//     group's score: the sum of its group_top largest c); the topk largest c
//     in open groups, falling, equal values in index order;
//     w = s[ids] (divided by their sum) * scale
//
// A wavefront per token.  Scores and choices are f64: which expert is chosen
// next to a border must not hang on the last bits of an f32 exponential, and
// a token's few hundred exponentials are hidden behind the launch.  A choice
// is compared as a 64-bit integer that orders like the f64 value, so one
// maximum over the wavefront is two DPP moves and a compare per step.
#include "qmm_device.hpp"
#include "qmm_internal.hpp"

namespace qmm {

namespace {

struct RouteArgs {
    const float *logits, *bias;
    int32_t *ids;
    float *weights;
    int64_t N;
    int E, groups, topk_groups, group_top, topk;
    bool sigmoid, renorm;
    double scale;
};

// An integer that orders like v; NaN counts as -inf; 0 is below everything.
__device__ __forceinline__ uint64_t order_key(double v) {
    if (v != v) v = -__builtin_inf();
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    return (b >> 63) ? ~b : (b | 0x8000000000000000ull);
}

template <int CTRL, int ROW_MASK, bool BOUND>
__device__ __forceinline__ uint64_t dpp_u64(uint64_t v) {
    const uint32_t lo = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)v, CTRL, ROW_MASK, 0xF, BOUND);
    const uint32_t hi = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)(v >> 32), CTRL, ROW_MASK, 0xF, BOUND);
    return ((uint64_t)hi << 32) | lo;
}
__device__ __forceinline__ uint64_t readlane_u64(uint64_t v, int lane) {
    const uint32_t lo = __builtin_amdgcn_readlane((int)(uint32_t)v, lane);
    const uint32_t hi = __builtin_amdgcn_readlane((int)(uint32_t)(v >> 32), lane);
    return ((uint64_t)hi << 32) | lo;
}
__device__ __forceinline__ uint64_t max_u64(uint64_t a, uint64_t b) { return a > b ? a : b; }

// The wavefront's largest key, uniform (0, the identity, where DPP reads nothing).
__device__ __forceinline__ uint64_t wave_max_u64(uint64_t v) {
    v = max_u64(v, dpp_u64<0xB1, 0xF, true>(v));    // quad_perm 1,0,3,2
    v = max_u64(v, dpp_u64<0x4E, 0xF, true>(v));    // quad_perm 2,3,0,1
    v = max_u64(v, dpp_u64<0x141, 0xF, true>(v));   // row_half_mirror
    v = max_u64(v, dpp_u64<0x140, 0xF, true>(v));   // row_mirror
    v = max_u64(v, dpp_u64<0x142, 0xA, false>(v));  // row_bcast15
    v = max_u64(v, dpp_u64<0x143, 0xC, false>(v));  // row_bcast31
    return readlane_u64(v, 63);
}
__device__ __forceinline__ double wave_sum_d(double v) {
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o, 64);
    return v;
}

// EPL experts per lane: expert e = 64 i + lane.  One wavefront per token,
// blockDim.x / 64 tokens per workgroup.
template <int EPL>
__global__ void __launch_bounds__(256) route_kernel(const RouteArgs a) {
    extern __shared__ double lds[];
    const int lane = (int)threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int64_t n = (int64_t)blockIdx.x * (blockDim.x >> 6) + wave;
    const bool grouped = a.groups > a.topk_groups;  // else every group stays open
    double *ss = lds + (size_t)wave * (64 * EPL + (grouped ? 64 * EPL + a.groups : 0));
    double *cs = ss + 64 * EPL, *gs = cs + 64 * EPL;  // grouped only
    const bool live = n < a.N;                         // uniform per wavefront

    float l[EPL];
    float best = -__builtin_inff();
#pragma unroll
    for (int i = 0; i < EPL; i++) {
        const int e = 64 * i + lane;
        float v = (live && e < a.E) ? a.logits[n * a.E + e] : -__builtin_inff();
        if (v != v) v = -__builtin_inff();             // NaN: masked
        l[i] = fminf(v, __FLT_MAX__);                  // +inf counts as the largest finite value
        best = fmaxf(best, l[i]);
    }
    double s[EPL], c[EPL];
    if (a.sigmoid) {
#pragma unroll
        for (int i = 0; i < EPL; i++) s[i] = 1.0 / (1.0 + exp(-(double)l[i]));
    } else {
#pragma unroll
        for (int o = 32; o > 0; o >>= 1) best = fmaxf(best, __shfl_xor(best, o, 64));
        double sum = 0.0;
#pragma unroll
        for (int i = 0; i < EPL; i++) {
            // a row with nothing left has no scores
            s[i] = best == -__builtin_inff() ? 0.0 : exp((double)l[i] - (double)best);
            sum += s[i];
        }
        sum = wave_sum_d(sum);
#pragma unroll
        for (int i = 0; i < EPL; i++) s[i] = sum > 0.0 ? s[i] / sum : 0.0;
    }
    uint64_t key[EPL];
#pragma unroll
    for (int i = 0; i < EPL; i++) {
        const int e = 64 * i + lane;
        c[i] = s[i] + ((a.bias && e < a.E) ? (double)a.bias[e] : 0.0);
        key[i] = e < a.E ? order_key(c[i]) : 0;
        ss[e] = s[i];
    }
    if (grouped) {
#pragma unroll
        for (int i = 0; i < EPL; i++) cs[64 * i + lane] = c[i] != c[i] ? -__builtin_inf() : c[i];
        __syncthreads();
        const int gsz = a.E / a.groups;
        for (int g = lane; g < a.groups; g += 64) {
            double m1 = -__builtin_inf(), m2 = -__builtin_inf();
            for (int j = 0; j < gsz; j++) {
                const double v = cs[g * gsz + j];
                m2 = v > m1 ? m1 : (v > m2 ? v : m2);
                m1 = v > m1 ? v : m1;
            }
            const double v = a.group_top == 2 ? m1 + m2 : m1;
            gs[g] = v != v ? -__builtin_inf() : v;
        }
        __syncthreads();
        // a group stays open if fewer than topk_groups groups come before it
#pragma unroll
        for (int i = 0; i < EPL; i++) {
            const int e = 64 * i + lane, g = e / gsz;
            if (e < a.E) {
                const double mine = gs[g];
                int before = 0;
                for (int o = 0; o < a.groups; o++) before += (gs[o] > mine || (gs[o] == mine && o < g)) ? 1 : 0;
                if (before >= a.topk_groups) key[i] = 0;
            }
        }
    } else {
        __syncthreads();  // ss
    }
    // the largest key, topk times; equal keys: the smallest index
    int chosen = 0;  // lane k: the k-th expert
    for (int k = 0; k < a.topk; k++) {
        uint64_t mine = 0;
#pragma unroll
        for (int i = 0; i < EPL; i++) mine = max_u64(mine, key[i]);
        const uint64_t top = wave_max_u64(mine);
        int e = -1;
#pragma unroll
        for (int i = EPL - 1; i >= 0; i--) {
            const uint64_t at = __ballot(key[i] == top);
            if (at) e = 64 * i + __ffsll((unsigned long long)at) - 1;
        }
        if (lane == k) chosen = e;
#pragma unroll
        for (int i = 0; i < EPL; i++)
            if (e == 64 * i + lane) key[i] = 0;
    }
    double w = lane < a.topk ? ss[chosen] : 0.0;
    if (a.renorm) {
        const double sum = wave_sum_d(w);
        w = sum > 0.0 ? w / sum : 0.0;
    }
    if (live && lane < a.topk) {
        a.ids[n * a.topk + lane] = chosen;
        a.weights[n * a.topk + lane] = (float)(w * a.scale);
    }
}

}  // namespace

hipError_t launch_moe_route(const float *logits, const float *bias, int64_t N, int64_t E, bool sigmoid, int64_t groups,
                            int64_t topk_groups, int group_top, int64_t topk, bool renorm, float scale, int32_t *ids,
                            float *weights, hipStream_t st) {
    RouteArgs a;
    a.logits = logits;
    a.bias = bias;
    a.ids = ids;
    a.weights = weights;
    a.N = N;
    a.E = (int)E;
    a.groups = (int)groups;
    a.topk_groups = (int)topk_groups;
    a.group_top = group_top;
    a.topk = (int)topk;
    a.sigmoid = sigmoid;
    a.renorm = renorm;
    a.scale = (double)scale;
    const int epl = E <= 64 ? 1 : E <= 128 ? 2 : E <= 256 ? 4 : E <= 512 ? 8 : 16;
    // four tokens per workgroup while their scores stay below 64 KB of LDS
    const unsigned wpb = epl > 4 ? 1 : (N >= 4 ? 4 : (unsigned)N);
    const size_t lds = 8 * (size_t)wpb * (64 * epl + (groups > topk_groups ? 64 * epl + groups : 0));
    const dim3 grid((unsigned)((N + wpb - 1) / wpb)), block(64 * wpb);
    switch (epl) {
    case 1: hipLaunchKernelGGL((route_kernel<1>), grid, block, lds, st, a); break;
    case 2: hipLaunchKernelGGL((route_kernel<2>), grid, block, lds, st, a); break;
    case 4: hipLaunchKernelGGL((route_kernel<4>), grid, block, lds, st, a); break;
    case 8: hipLaunchKernelGGL((route_kernel<8>), grid, block, lds, st, a); break;
    default: hipLaunchKernelGGL((route_kernel<16>), grid, block, lds, st, a); break;
    }
    return hipGetLastError();
}

}  // namespace qmm
