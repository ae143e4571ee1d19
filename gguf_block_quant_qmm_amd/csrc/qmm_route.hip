// qmm_route.hip -- routing of tokens to experts (include/qmm.h, qmm_moe_route):
//     s = softmax(l) or sigmoid(l);  c = s + bias
//     the topk_groups groups with the largest group scores stay open (a
//     group's score: the sum of its group_top largest c); the topk largest c
//     in open groups, falling, equal values in index order;
//     w = s[ids] (divided by their sum) * scale
//
// A wavefront per token.  Scores and choices are f64: which expert is chosen
// next to a border must not hang on the last bits of an f32 exponential, and
// a token's few hundred exponentials are hidden behind the launch.  The
// running choices are f64 values with NaN for an expert that is out (chosen, or
// in a closed group): v_max_f64 passes over NaN, so a maximum over the
// wavefront is two DPP moves and one instruction per step.
//
// Bound by the chain of topk maxima, each waiting for the one before it: 1 token,
// 8 of 64 experts, 3.3 us (a launch's start).  4096 tokens, 256 experts in groups,
// sigmoid scores: 11.4 us, against 1 us of memory time for 4 MB of logits; issuing
// the VALU instructions alone takes 7.7, more where they are f64.  512 tokens, 8 of
// 64, softmax: 5.0.  Profiler's medians.
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

template <int CTRL, int ROW_MASK>
__device__ __forceinline__ double dpp_max(double v) {
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    // lanes without a source keep their own value
    const uint32_t lo = __builtin_amdgcn_update_dpp((int)(uint32_t)b, (int)(uint32_t)b, CTRL, ROW_MASK, 0xF, false);
    const uint32_t hi = __builtin_amdgcn_update_dpp((int)(uint32_t)(b >> 32), (int)(uint32_t)(b >> 32), CTRL, ROW_MASK, 0xF, false);
    return fmax(v, __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo));
}
// The wavefront's largest value (NaN only if all are), uniform.
__device__ __forceinline__ double wave_max_d(double v) {
    v = dpp_max<0xB1, 0xF>(v);   // quad_perm 1,0,3,2
    v = dpp_max<0x4E, 0xF>(v);   // quad_perm 2,3,0,1
    v = dpp_max<0x141, 0xF>(v);  // row_half_mirror
    v = dpp_max<0x140, 0xF>(v);  // row_mirror
    v = dpp_max<0x142, 0xA>(v);  // row_bcast15
    v = dpp_max<0x143, 0xC>(v);  // row_bcast31: the maximum, in lane 63
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = __builtin_amdgcn_readlane((int)(uint32_t)b, 63);
    const uint32_t hi = __builtin_amdgcn_readlane((int)(uint32_t)(b >> 32), 63);
    return __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
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
    double *ss = lds + (size_t)wave * (64 * EPL + (grouped ? 64 * EPL + 2 * a.groups : 0));
    double *cs = ss + 64 * EPL, *gs = cs + 64 * EPL, *gopen = gs + a.groups;  // grouped only
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
    const double out = __builtin_nan("");
#pragma unroll
    for (int i = 0; i < EPL; i++) {
        const int e = 64 * i + lane;
        c[i] = s[i] + ((a.bias && e < a.E) ? (double)a.bias[e] : 0.0);
        if (c[i] != c[i]) c[i] = -__builtin_inf();
        ss[e] = s[i];
        if (grouped) cs[e] = c[i];
        if (e >= a.E) c[i] = out;
    }
    __syncthreads();
    if (grouped) {
        // group g on the 64 / groups (a power of two) lanes g * parts ..: each
        // scans every parts-th expert for its two largest, then they merge
        const int gsz = a.E / a.groups;
        int parts = 1;
        while (2 * parts * a.groups <= 64) parts *= 2;
        for (int g0 = 0; g0 < a.groups; g0 += 64) {
            const int g = g0 + lane / parts, part = lane % parts;
            double m1 = -__builtin_inf(), m2 = -__builtin_inf();
            if (g < a.groups) {
                for (int j = part; j < gsz; j += parts) {
                    const double v = cs[g * gsz + j];
                    m2 = fmax(m2, fmin(m1, v));
                    m1 = fmax(m1, v);
                }
            }
            for (int o = 1; o < parts; o *= 2) {
                const double n1 = __shfl_xor(m1, o, 64), n2 = __shfl_xor(m2, o, 64);
                m2 = fmax(fmin(m1, n1), fmax(m2, n2));
                m1 = fmax(m1, n1);
            }
            if (g < a.groups && part == 0) {
                const double v = a.group_top == 2 ? m1 + m2 : m1;
                gs[g] = v != v ? -__builtin_inf() : v;
            }
        }
        __syncthreads();
        // a group stays open if fewer than topk_groups groups come before it;
        // a closed one is marked by a NaN where its score was
        for (int g0 = 0; g0 < a.groups; g0 += 64) {
            const int g = g0 + lane;
            int before = 0;
            if (g < a.groups) {
                const double mine = gs[g];
                for (int o = 0; o < a.groups; o++) before += (gs[o] > mine || (gs[o] == mine && o < g)) ? 1 : 0;
            }
            if (g < a.groups) gopen[g] = before < a.topk_groups ? 0.0 : out;
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < EPL; i++) {
            const int e = 64 * i + lane;
            if (e < a.E && gopen[e / gsz] != 0.0) c[i] = out;
        }
    }
    // the largest choice, topk times; equal ones: the smallest index
    int chosen = 0;  // lane k: the k-th expert
    for (int k = 0; k < a.topk; k++) {
        double mine = c[0];
#pragma unroll
        for (int i = 1; i < EPL; i++) mine = fmax(mine, c[i]);
        const double top = wave_max_d(mine);
        int e = 0;
#pragma unroll
        for (int i = EPL - 1; i >= 0; i--) {
            const uint64_t at = __ballot(c[i] == top);
            if (at) e = 64 * i + __ffsll((unsigned long long)at) - 1;
        }
        if (lane == k) chosen = e;
#pragma unroll
        for (int i = 0; i < EPL; i++)
            if (e == 64 * i + lane) c[i] = out;
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
                            int64_t topk_groups, int group_top, int64_t topk, bool renorm, double scale, int32_t *ids,
                            float *weights, hipStream_t st) {
    const int epl = E <= 64 ? 1 : E <= 128 ? 2 : E <= 256 ? 4 : E <= 512 ? 8 : 16;
    // a grid holds fewer than 2^32 threads: at most 2^25 tokens per launch
    constexpr int64_t kTokens = int64_t(1) << 25;
    for (int64_t n0 = 0; n0 < N; n0 += kTokens) {
        RouteArgs a;
        a.logits = logits + n0 * E;
        a.bias = bias;
        a.ids = ids + n0 * topk;
        a.weights = weights + n0 * topk;
        a.N = N - n0 < kTokens ? N - n0 : kTokens;
        a.E = (int)E;
        a.groups = (int)groups;
        a.topk_groups = (int)topk_groups;
        a.group_top = group_top;
        a.topk = (int)topk;
        a.sigmoid = sigmoid;
        a.renorm = renorm;
        a.scale = scale;
        // four tokens per workgroup while their scores stay below 64 KB of LDS
        const unsigned wpb = epl > 4 ? 1 : (a.N >= 4 ? 4 : (unsigned)a.N);
        const size_t lds = 8 * (size_t)wpb * (64 * epl + (groups > topk_groups ? 64 * epl + 2 * groups : 0));
        const dim3 grid((unsigned)((a.N + wpb - 1) / wpb)), block(64 * wpb);
        switch (epl) {
        case 1: hipLaunchKernelGGL((route_kernel<1>), grid, block, lds, st, a); break;
        case 2: hipLaunchKernelGGL((route_kernel<2>), grid, block, lds, st, a); break;
        case 4: hipLaunchKernelGGL((route_kernel<4>), grid, block, lds, st, a); break;
        case 8: hipLaunchKernelGGL((route_kernel<8>), grid, block, lds, st, a); break;
        default: hipLaunchKernelGGL((route_kernel<16>), grid, block, lds, st, a); break;
        }
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace qmm
