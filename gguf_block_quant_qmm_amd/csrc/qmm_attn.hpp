// qmm_attn.hpp -- what the two forms of attention over the paged cache share:
// which tokens a row sees, how the tokens are shared out over workgroups, the
// rows' f16 parts.  Included only by the HIP sources of attention.
#pragma once

#include "qmm_internal.hpp"
#include "qmm_kv.hpp"

namespace qmm {

struct AttnArgs {
    const float *Q;
    float *out;
    float *part;   // [rows][Hq][splits][D]: sum of p * value under the split's maximum
    float2 *stat;  // [rows][Hq][splits]: (maximum, sum of p); -inf: the split saw nothing
    int64_t q_stride, window, block0;
    float scale, softcap;
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
    int64_t lo_any, hi_any;  // seen by some row of the tile: lo_any <= j < hi_any
    int64_t lo_all, hi_all;  // seen by every row (where the pages exist)
    int64_t k0, k1;
};

__device__ __forceinline__ void attn_sees(const AttnArgs &a, const KvNew &nw, int t, int64_t &lo, int64_t &hi) {
    const int64_t i = nw.index + t, cap = (int64_t)a.kv.max_pages << a.kv.page_shift;
    hi = a.causal && i + 1 < nw.len ? i + 1 : nw.len;
    hi = hi < cap ? hi : cap;
    hi = hi > 0 ? hi : 0;
    lo = a.window && i - a.window + 1 > 0 ? i - a.window + 1 : 0;
    lo = lo < hi ? lo : hi;
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
    int64_t lo1, hi1;
    attn_sees(a, w.nw, w.r0 / a.G, w.lo_any, w.hi_all);
    attn_sees(a, w.nw, (w.r0 + w.nrows - 1) / a.G, lo1, hi1);
    w.hi_any = hi1;
    w.lo_all = lo1;
    const int64_t c0 = w.lo_any / CH, c1 = (w.hi_any + CH - 1) / CH;
    int64_t per = (c1 - c0 + a.splits - 1) / a.splits;
    per = per > least ? per : least;
    const int64_t b0 = c0 + per * w.split, b1 = b0 + per;
    w.k0 = b0 * CH;
    w.k1 = (b1 < c1 ? b1 : c1) * CH;
    return true;
}

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

constexpr float kLog2e = 1.44269504088896340736f;

// Scores in base 2 from the raw products: mul is scale * 2^-e * log2(e), or,
// under a softcap, scale * 2^-e / softcap.
__device__ __forceinline__ float attn_score(float raw, float mul, float softcap) {
    return softcap > 0.f ? softcap * kLog2e * tanhf(raw * mul) : raw * mul;
}
__device__ __forceinline__ float attn_mul(const AttnArgs &a, int e) {
    return ldexpf(a.softcap > 0.f ? a.scale / a.softcap : a.scale * kLog2e, -e);
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
