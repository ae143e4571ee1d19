// qmm_attn.hpp -- what the two forms of attention over the paged cache share:
// which tokens a row sees, how the tokens are shared out over workgroups, the
// rows' f16 parts.  Included only by the HIP sources of attention.
#pragma once

#include <float.h>

#include "qmm_internal.hpp"
#include "qmm_kv.hpp"

namespace qmm {

struct AttnArgs {
    const float *Q;
    float *out;
    float *part;   // [rows][Hq][splits][D]: sum of p * value under the split's maximum
    float2 *stat;  // [rows][Hq][splits]: (maximum, sum of p); -inf: the split saw nothing
    int64_t q_stride, window, block0;
    float mul;    // mul * 2^mul_exp: scale in base 2
    int mul_exp;
    float cap, cap_inv, cap_from, cap_rate;  // of cap_scores; cap 0: none
    int Hq, G, splits, tiles;
    bool causal;
    KvArgs kv;
};

// A workgroup's share: query rows r0 .. r0 + RT - 1 of a key-value head of a
// sequence (row r is new token r / G with query head h * G + r % G), tokens
// k0 .. k1 - 1 in whole chunks.  The unit (sequence, head) runs fastest over the
// workgroups, so with a multiple of 8 of them a unit's workgroups share an XCD's L2;
// the last row tiles, with the most to see, start first.
struct AttnShare {
    KvNew nw;
    int s, h, split, r0, nrows;
    int lo_any, hi_any;  // seen by some row of the tile: lo_any <= j < hi_any
    int lo_all, hi_all;  // seen by every row (where the pages exist)
    int k0, k1;
};

// What new token t sees: lo <= j < hi.  A table reaches no further than token 2^30.
__device__ __forceinline__ void attn_sees(const AttnArgs &a, const KvNew &nw, int t, int &lo, int &hi) {
    const int64_t i = nw.index + t, cap = (int64_t)a.kv.max_pages << a.kv.page_shift;
    int64_t to = a.causal && i + 1 < nw.len ? i + 1 : nw.len;
    to = to < cap ? to : cap;
    hi = (int)(to > 0 ? to : 0);
    const int64_t from = a.window && i - a.window + 1 > 0 ? i - a.window + 1 : 0;
    lo = (int)(from < hi ? from : hi);
}

// False if the workgroup has no rows.  CH: tokens of a chunk; a split takes at
// least `least` chunks.
template <int RT, int CH>
__device__ __forceinline__ bool attn_share(const AttnArgs &a, int least, AttnShare &w) {
    const uint32_t units = (uint32_t)a.kv.seqs * (uint32_t)a.kv.heads;
    const int64_t b = a.block0 + blockIdx.x;
    uint32_t u, j;
    if (b <= UINT32_MAX) {
        j = (uint32_t)b / units;
        u = (uint32_t)b - j * units;
    } else {
        j = (uint32_t)(b / units);
        u = (uint32_t)(b - (int64_t)j * units);
    }
    w.s = (int)(u / (uint32_t)a.kv.heads);
    w.h = (int)(u - (uint32_t)w.s * (uint32_t)a.kv.heads);
    const uint32_t tile = j / (uint32_t)a.splits;
    w.split = (int)(j - tile * (uint32_t)a.splits);
    w.nw = kv_new(a.kv, w.s);
    const int64_t r0 = (int64_t)(a.tiles - 1 - (int)tile) * RT, rows = (int64_t)w.nw.count * a.G;
    if (r0 >= rows) return false;
    w.r0 = (int)r0;
    w.nrows = (int)(rows - r0 < RT ? rows - r0 : RT);
    int lo1, hi1;
    attn_sees(a, w.nw, w.r0 / a.G, w.lo_any, w.hi_all);
    attn_sees(a, w.nw, (w.r0 + w.nrows - 1) / a.G, lo1, hi1);
    w.hi_any = hi1;
    w.lo_all = lo1;
    const int c0 = w.lo_any / CH, c1 = (w.hi_any + CH - 1) / CH;
    int per = (c1 - c0 + a.splits - 1) / a.splits;
    per = per > least ? per : least;
    const int64_t b0 = c0 + (int64_t)per * w.split, b1 = b0 + per;
    w.k0 = (int)(b0 < c1 ? b0 : c1) * CH;
    w.k1 = (int)(b1 < c1 ? b1 : c1) * CH;
    return true;
}

// A sequence's row of the page table; token i's page, or -1.  i >= 0; the kernels ask up to 300 tokens past a
// sequence's end, so past the 2^30 of the longest table too.
struct Pages {
    const int32_t *row;
    int shift, columns, pages;
    __device__ __forceinline__ Pages(const AttnArgs &a, int s)
        : row(a.kv.table + (int64_t)s * a.kv.table_stride), shift(a.kv.page_shift), columns(a.kv.max_pages), pages(a.kv.pages) {}
    __device__ __forceinline__ int operator()(int i) const {
        const int c = i >> shift;
        const int p = c < columns ? row[c] : -1;
        return (uint32_t)p < (uint32_t)pages ? p : -1;
    }
};

// The value of the other half of the wavefront (lane ^ 32), and of the neighbouring row of
// 16 lanes (lane ^ 16), folded into v by `op`.
template <typename F>
__device__ __forceinline__ float fold32(float v, F op) {
    const auto r = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(uint32_t, v), __builtin_bit_cast(uint32_t, v), false, false);
    const uint32_t x = r[0], y = r[1];  // a bit cast of r[1] itself reads element 0
    return op(__builtin_bit_cast(float, x), __builtin_bit_cast(float, y));
}
template <typename F>
__device__ __forceinline__ float fold16(float v, F op) {
    const auto r = __builtin_amdgcn_permlane16_swap(__builtin_bit_cast(uint32_t, v), __builtin_bit_cast(uint32_t, v), false, false);
    const uint32_t x = r[0], y = r[1];  // a bit cast of r[1] itself reads element 0
    return op(__builtin_bit_cast(float, x), __builtin_bit_cast(float, y));
}
struct MaxOp {
    __device__ __forceinline__ float operator()(float x, float y) const { return fmaxf(x, y); }
};
struct SumOp {
    __device__ __forceinline__ float operator()(float x, float y) const { return x + y; }
};

// The power of two under which a query row is split in two f16 parts: its
// largest |value| comes to 2^14 .. 2^15.
__device__ __forceinline__ int row_exponent(float amax) {
    if (!(amax > 0.f) || !__builtin_isfinite(amax)) return 0;
    const int e = 15 - __builtin_amdgcn_frexp_expf(amax);
    return e < 126 ? e : 126;
}

// A raw product (queries times 2^e) times this is the score in base 2.  Finite: a product of 0 has a score of 0.
__device__ __forceinline__ float attn_mul(const AttnArgs &a, int e) {
    return fminf(fmaxf(ldexpf(a.mul, a.mul_exp - e), -FLT_MAX), FLT_MAX);
}

// Scores t in base 2 under a softcap (c in base 2): c tanh(t / c).  Below c / 2: t (1 + P(t^2 / c^2)), which keeps the
// bits of a score far below the cap; else c (1 - 2 / (e^(2t/c) + 1)).  Within 2^-21 of the capped score either
// way, where the second alone would be 2^-22 of the cap and faster in prompts (512 tokens over 4096, 32/8 heads
// of 128 f16: 98 us, 90 so, 81 without a cap; of 64: 73, 62, 52).  P is fitted to tanh(x) / x - 1 for the least
// largest error of tanh, 2^-26, and in the unit of x that leaves its leading coefficient 1: the constants are
// then literals and hold no registers through the main loop.  Both forms for every score: a branch that leaves
// the exponentials out costs registers that the kernels lack (it spills on Q8_0, calls without a cap too).
template <int N, typename S>
__device__ __forceinline__ void cap_scores(const AttnArgs &a, S &s) {
#pragma unroll
    for (int i = 0; i < N; i++) {
        const float t = s[i], x = t * a.cap_inv, z = x * x;
        const float near = t * fmaf(fmaf(fmaf(z - 1.11485296f, z, 1.01486586f), z, -0.919883146f), z, 1.f);
        const float far = a.cap * fmaf(-2.f, __builtin_amdgcn_rcpf(__builtin_amdgcn_exp2f(t * a.cap_rate) + 1.f), 1.f);
        s[i] = fabsf(t) < a.cap_from ? near : far;
        if (i % 4 == 3) __builtin_amdgcn_sched_barrier(0);  // four at a time
    }
}

// p = hi + lo in f16 to 2^-23 of p (2^-25 near 0): two conversions for two values and one FMA
// that reads its f16 operand as it is for each rest (p - hi, exact).  minus_one is
// -1 where the compiler cannot see it: it would convert and subtract instead.
__device__ __forceinline__ float opaque_minus_one() {
    float v = -1.f;
    asm("" : "+s"(v));
    return v;
}
__device__ __forceinline__ void split2(float p0, float p1, float minus_one, half2_t &hi, half2_t &lo) {
    typedef float float2_t __attribute__((ext_vector_type(2)));
    hi = __builtin_convertvector((float2_t{p0, p1}), half2_t);
    const float r0 = fmaf((float)hi.x, minus_one, p0), r1 = fmaf((float)hi.y, minus_one, p1);
    lo = __builtin_convertvector((float2_t{r0, r1}), half2_t);
}

// Four codes of a dword as f16 pairs, exactly: byte ^ 0x80 is code + 128, under
// the high byte of 1024 it reads 1152 + code.
__device__ __forceinline__ half4 codes4(uint32_t v) {
    const uint32_t u = v ^ 0x80808080u;
    const half2_t off = {(_Float16)1152.f, (_Float16)1152.f};
    const half2_t a = __builtin_bit_cast(half2_t, __builtin_amdgcn_perm(0x64646464u, u, 0x04010400u)) - off;
    const half2_t b = __builtin_bit_cast(half2_t, __builtin_amdgcn_perm(0x64646464u, u, 0x04030402u)) - off;
    return half4{a.x, a.y, b.x, b.y};
}
__device__ __forceinline__ half8 codes8(u32x2_t v) {
    const half4 a = codes4(v.x), b = codes4(v.y);
    return half8{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
}

// The form for many rows (qmm_attn_prompt.hip): rows of a workgroup, tokens of a tile.
constexpr int kPromptRows = 128, kPromptChunk = 64;
hipError_t launch_attn_prompt(const AttnArgs &a, int dtype, int D, int64_t blocks, hipStream_t st);

}  // namespace qmm
