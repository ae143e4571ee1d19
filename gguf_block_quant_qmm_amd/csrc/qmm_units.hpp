// qmm_units.hpp -- the f32 arithmetic of one 64-weight unit of every block
// format (GEMV family), the generic per-block dot products, and the Q8_0
// quantizer's block arithmetic: device code shared by the decode GEMVs, the
// routed experts' products and the block norm.
#pragma once

#include "qmm_device.hpp"

namespace qmm {

__device__ __forceinline__ float fma_h(_Float16 h, float x, float acc) { return fmaf((float)h, x, acc); }


// ----------------------------------------------------------------- units ----
// A unit is 64 weights of one row.  Q8_0/Q4_0: a pair of consecutive blocks
// (an even number of blocks per row keeps every pair dword aligned).  Q4_K:
// one 64-weight chunk of a super-block (sub-blocks 2c and 2c+1).  Q6_K: the 64
// weights {128h + 32g + 16lh + i : g < 4, i < 16} of one super-block, which
// share one 16-byte slice of each ql half and of qh.
//   Off          per-lane byte offsets inside a row (computed once)
//   load(row,o)  the unit's raw dwords (row pointer uniform across the wave)
//   x4(u, i)     float4 index of local activations 4i..4i+3 of unit u
//   dot(v,x,o)   the unit's dot product, f32

template <int DT> struct Unit;

// 4-bit codes enter the f32 arithmetic (v_fma_mix_f32) as f16 subnormals: a
// dword masked with 0x000F000F holds two codes c as c * 2^-24, masked with
// 0x00F000F0 as c * 2^-20 -- one VOP2 instruction per two codes, exact.  Every
// weight is formed exactly (Q4_0, Q8_0, Q6_K) or with one rounding (Q4_K)
// before it meets its activation, so the usual f32 dot-product error bound
// relative to sum |w x| holds: no offset is ever taken out through a sum of
// activations (that would cancel when the weights do).
__device__ __forceinline__ half2_t as_h2(uint32_t v) { return __builtin_bit_cast(half2_t, v); }

constexpr float TWO24 = 16777216.0f, TWO20 = 1048576.0f;

template <> struct Unit<QMM_Q4_0> {
    static constexpr int NL = 9;
    struct Off { uint32_t a; };
    __device__ static Off lane_off(int u) { return {36u * u}; }
    __device__ static void load(Rsrc rs, uint32_t row, const Off &o, uint32_t (&v)[NL]) { ldb(rs, o.a, row, v); }
    __device__ static int x4(int u, int i) { return 16 * u + i; }
    __device__ static float dot(const uint32_t (&v)[NL], const float (&xv)[64], const Off &) {
        // The unit is two blocks, 36 bytes: d0 qs0[16] d1 qs1[16].  Block 0's
        // codes sit in dwords [qs0 qs1 qs14 qs15] (realigned from v0, v4) and
        // v1..v3 = qs2..13; block 1's in v5..v8.  Element e < 16 is the low
        // nibble of qs[e], element e + 16 its high nibble.  Low nibbles become
        // (q - 8) 2^-24, high nibbles (q - 8) 2^-20: exact f16 subnormals.
        const half2_t b24 = as_h2(0x80088008u), b20 = as_h2(0x80808080u);  // -8 * 2^-24, -128 * 2^-24
        const uint32_t D[2][4] = {{__builtin_amdgcn_alignbyte(v[4], v[0], 2), v[1], v[2], v[3]},
                                  {v[5], v[6], v[7], v[8]}};
        float lo[2][2], hi[2][2];
#pragma unroll
        for (int b = 0; b < 2; b++) {
            const float *xb = xv + 32 * b;
#pragma unroll
            for (int i = 0; i < 4; i++) {
                // qs index of the dword's bytes 0..3
                const int e0 = b == 1 ? 4 * i : (i == 0 ? 0 : 4 * i - 2);
                const int e1 = e0 + 1;
                const int e2 = (b == 0 && i == 0) ? 14 : e0 + 2, e3 = e2 + 1;
                const uint32_t d = D[b][i], t = d >> 8;
                const half2_t p0 = as_h2(d & 0x000F000Fu) + b24, p1 = as_h2(d & 0x00F000F0u) + b20;
                const half2_t p2 = as_h2(t & 0x000F000Fu) + b24, p3 = as_h2(t & 0x00F000F0u) + b20;
                const int c = i & 1;
                float l = i < 2 ? 0.f : lo[b][c], h = i < 2 ? 0.f : hi[b][c];
                l = fma_h(p0.x, xb[e0], l); h = fma_h(p1.x, xb[16 + e0], h);
                l = fma_h(p0.y, xb[e2], l); h = fma_h(p1.y, xb[16 + e2], h);
                l = fma_h(p2.x, xb[e1], l); h = fma_h(p3.x, xb[16 + e1], h);
                l = fma_h(p2.y, xb[e3], l); h = fma_h(p3.y, xb[16 + e3], h);
                lo[b][c] = l; hi[b][c] = h;
            }
        }
        const float s0 = fmaf(lo[0][0] + lo[0][1], TWO24, (hi[0][0] + hi[0][1]) * TWO20);
        const float s1 = fmaf(lo[1][0] + lo[1][1], TWO24, (hi[1][0] + hi[1][1]) * TWO20);
        return fmaf(h2f(v[4] >> 16), s1, h2f(v[0]) * s0);
    }
};

template <> struct Unit<QMM_Q4_1> {
    // The unit is two 20-byte blocks (d, m, qs[16]) -- every dword aligned:
    // v0 = d0|m0, v1..v4 = qs0[0..16), v5 = d1|m1, v6..v9 = qs1.  Codes enter
    // as exact f16 subnormals (low nibbles c 2^-24, high nibbles c 2^-20); each
    // weight d*q + m is formed with one rounding (v_fma_mix_f32 with d*2^24 or
    // d*2^20 and m), then multiplied into x with an f32 FMA -- as for Q4_K.
    static constexpr int NL = 10;
    struct Off { uint32_t a; };
    __device__ static Off lane_off(int u) { return {40u * u}; }
    __device__ static void load(Rsrc rs, uint32_t row, const Off &o, uint32_t (&v)[NL]) { ldb(rs, o.a, row, v); }
    __device__ static int x4(int u, int i) { return 16 * u + i; }
    __device__ static float dot(const uint32_t (&v)[NL], const float (&xv)[64], const Off &) {
        float acc[4];
#pragma unroll
        for (int b = 0; b < 2; b++) {
            const float d = h2f(v[5 * b]), m = h2f(v[5 * b] >> 16);
            const float s24 = d * TWO24, s20 = d * TWO20;
            const float *xb = xv + 32 * b;
            float l = 0.f, h = 0.f;
#pragma unroll
            for (int i = 0; i < 4; i++) {
                // qs[4i .. 4i+4): elements 4i..4i+3 (low nibbles), 16+4i.. (high)
                const uint32_t dw = v[5 * b + 1 + i], t = dw >> 8;
                const half2_t p0 = as_h2(dw & 0x000F000Fu), p1 = as_h2(dw & 0x00F000F0u);
                const half2_t p2 = as_h2(t & 0x000F000Fu), p3 = as_h2(t & 0x00F000F0u);
                l = fmaf(fma_h(p0.x, s24, m), xb[4 * i], l);     h = fmaf(fma_h(p1.x, s20, m), xb[16 + 4 * i], h);
                l = fmaf(fma_h(p0.y, s24, m), xb[4 * i + 2], l); h = fmaf(fma_h(p1.y, s20, m), xb[16 + 4 * i + 2], h);
                l = fmaf(fma_h(p2.x, s24, m), xb[4 * i + 1], l); h = fmaf(fma_h(p3.x, s20, m), xb[16 + 4 * i + 1], h);
                l = fmaf(fma_h(p2.y, s24, m), xb[4 * i + 3], l); h = fmaf(fma_h(p3.y, s20, m), xb[16 + 4 * i + 3], h);
            }
            acc[2 * b] = l;
            acc[2 * b + 1] = h;
        }
        return (acc[0] + acc[1]) + (acc[2] + acc[3]);
    }
};
template <> struct Unit<QMM_Q8_0> {
    static constexpr int NL = 17;
    struct Off { uint32_t a; };
    __device__ static Off lane_off(int u) { return {68u * u}; }
    __device__ static void load(Rsrc rs, uint32_t row, const Off &o, uint32_t (&v)[NL]) { ldb(rs, o.a, row, v); }
    __device__ static int x4(int u, int i) { return 16 * u + i; }
    __device__ static float dot(const uint32_t (&v)[NL], const float (&xv)[64], const Off &) {
        const half2_t bias = {(_Float16)-1152.0f, (_Float16)-1152.0f};  // (q + 128) - 128
        float blk[2];
#pragma unroll
        for (int b = 0; b < 2; b++) {
            half2_t w[8][2];  // [dword][p02, p13]
#pragma unroll
            for (int i = 0; i < 8; i++) {
                const uint32_t q = (b == 0 ? __builtin_amdgcn_alignbyte(v[i + 1], v[i], 2) : v[9 + i]) ^ 0x80808080u;
                w[i][0] = bytes02_as_f16(q) + bias; w[i][1] = bytes13_as_f16(q) + bias;
            }
            const float *xb = xv + 32 * b;
            float s8[8];
#pragma unroll
            for (int i = 0; i < 8; i++) s8[i] = fma_h(w[i][0].x, xb[4 * i], 0.f);
#pragma unroll
            for (int i = 0; i < 8; i++) s8[i] = fma_h(w[i][1].x, xb[4 * i + 1], s8[i]);
#pragma unroll
            for (int i = 0; i < 8; i++) s8[i] = fma_h(w[i][0].y, xb[4 * i + 2], s8[i]);
#pragma unroll
            for (int i = 0; i < 8; i++) s8[i] = fma_h(w[i][1].y, xb[4 * i + 3], s8[i]);
            blk[b] = ((s8[0] + s8[1]) + (s8[2] + s8[3])) + ((s8[4] + s8[5]) + (s8[6] + s8[7]));
        }
        return fmaf(h2f(v[8] >> 16), blk[1], h2f(v[0]) * blk[0]);
    }
};

template <> struct Unit<QMM_Q4_K> {
    static constexpr int NL = 12;  // 4 header dwords (d, dmin, 12 scale bytes) + 8 nibble dwords
    struct Off { uint32_t hdr, qs; int c; };
    __device__ static Off lane_off(int u) {
        const uint32_t h = 144u * (u >> 2);
        return {h, h + 16u + 32u * (u & 3), u & 3};
    }
    __device__ static void load(Rsrc rs, uint32_t row, const Off &o, uint32_t (&v)[NL]) {
        uint32_t h[4], q[8];
        ldb(rs, o.hdr, row, h);
        ldb(rs, o.qs, row, q);
#pragma unroll
        for (int i = 0; i < 4; i++) v[i] = h[i];
#pragma unroll
        for (int i = 0; i < 8; i++) v[4 + i] = q[i];
    }

    __device__ static int x4(int u, int i) { return 16 * u + i; }
    __device__ static float dot(const uint32_t (&v)[NL], const float (&xv)[64], const Off &o) {
        // sub-block 2c = low nibbles of qs[32c + j], 2c+1 = high nibbles.  Each
        // weight d*sc*q - dmin*m is formed with one rounding (v_fma_mix_f32 of
        // the subnormal code c*2^-24 or c*2^-20 with d*sc*2^24 or d*sc*2^20),
        // then multiplied into x with an f32 FMA.
        const float d = h2f(v[0]), dmin = h2f(v[0] >> 16);
        int sc0, m0, sc1, m1;
        q4k_scale_min(v[1], v[2], v[3], 2 * o.c, sc0, m0);
        q4k_scale_min(v[1], v[2], v[3], 2 * o.c + 1, sc1, m1);
        const float s0 = d * (float)sc0 * TWO24, n0 = -(dmin * (float)m0);
        const float s1 = d * (float)sc1 * TWO20, n1 = -(dmin * (float)m1);
        float acc[4];
#pragma unroll
        for (int i = 0; i < 8; i++) {
            const uint32_t dw = v[4 + i], t = dw >> 8;
            const half2_t p0 = as_h2(dw & 0x000F000Fu), p1 = as_h2(dw & 0x00F000F0u);
            const half2_t p2 = as_h2(t & 0x000F000Fu), p3 = as_h2(t & 0x00F000F0u);
            const int c = 2 * (i & 1);
            float l = i < 2 ? 0.f : acc[c], h = i < 2 ? 0.f : acc[c + 1];
            l = fmaf(fma_h(p0.x, s0, n0), xv[4 * i], l);     h = fmaf(fma_h(p1.x, s1, n1), xv[32 + 4 * i], h);
            l = fmaf(fma_h(p0.y, s0, n0), xv[4 * i + 2], l); h = fmaf(fma_h(p1.y, s1, n1), xv[32 + 4 * i + 2], h);
            l = fmaf(fma_h(p2.x, s0, n0), xv[4 * i + 1], l); h = fmaf(fma_h(p3.x, s1, n1), xv[32 + 4 * i + 1], h);
            l = fmaf(fma_h(p2.y, s0, n0), xv[4 * i + 3], l); h = fmaf(fma_h(p3.y, s1, n1), xv[32 + 4 * i + 3], h);
            acc[c] = l; acc[c + 1] = h;
        }
        return (acc[0] + acc[2]) + (acc[1] + acc[3]);
    }
};

template <> struct Unit<QMM_Q5_K> {
    // As Q4_K (unit = 64-weight chunk c of a super-block: sub-blocks 2c, 2c+1),
    // plus the fifth bit of every weight: bit i of qh[e] for element e of
    // sub-block i.  The bit joins the code while it is still an exact f16
    // subnormal: bit 4 of a low-nibble pair (c 2^-24), bit 8 of a high-nibble
    // pair (c 2^-20).  Super-blocks are 176 = 11 * 16 bytes: 16-byte aligned.
    static constexpr int NL = 20;  // 4 header dwords, 8 qh dwords, 8 nibble dwords
    struct Off { uint32_t hdr, qs; int c; };
    __device__ static Off lane_off(int u) {
        const uint32_t h = 176u * (u >> 2);
        return {h, h + 48u + 32u * (u & 3), u & 3};
    }
    __device__ static void load(Rsrc rs, uint32_t row, const Off &o, uint32_t (&v)[NL]) {
        uint32_t h[12], q[8];
        ldb(rs, o.hdr, row, h);  // d, dmin, scales, qh
        ldb(rs, o.qs, row, q);
#pragma unroll
        for (int i = 0; i < 12; i++) v[i] = h[i];
#pragma unroll
        for (int i = 0; i < 8; i++) v[12 + i] = q[i];
    }
    __device__ static int x4(int u, int i) { return 16 * u + i; }
    __device__ static float dot(const uint32_t (&v)[NL], const float (&xv)[64], const Off &o) {
        const float d = h2f(v[0]), dmin = h2f(v[0] >> 16);
        int sc0, m0, sc1, m1;
        q4k_scale_min(v[1], v[2], v[3], 2 * o.c, sc0, m0);
        q4k_scale_min(v[1], v[2], v[3], 2 * o.c + 1, sc1, m1);
        const float s0 = d * (float)sc0 * TWO24, n0 = -(dmin * (float)m0);
        const float s1 = d * (float)sc1 * TWO20, n1 = -(dmin * (float)m1);
        float acc[4];
#pragma unroll
        for (int i = 0; i < 8; i++) {
            const uint32_t dw = v[12 + i], t = dw >> 8;
            const uint32_t hq = v[4 + i] >> (2 * o.c), ht = hq >> 8;  // qh[4i .. 4i+4), bits 2c and 2c+1 at 0, 1
            const half2_t p0 = as_h2((dw & 0x000F000Fu) | ((hq << 4) & 0x00100010u));
            const half2_t p1 = as_h2((dw & 0x00F000F0u) | ((hq << 7) & 0x01000100u));
            const half2_t p2 = as_h2((t & 0x000F000Fu) | ((ht << 4) & 0x00100010u));
            const half2_t p3 = as_h2((t & 0x00F000F0u) | ((ht << 7) & 0x01000100u));
            const int c = 2 * (i & 1);
            float l = i < 2 ? 0.f : acc[c], h = i < 2 ? 0.f : acc[c + 1];
            l = fmaf(fma_h(p0.x, s0, n0), xv[4 * i], l);     h = fmaf(fma_h(p1.x, s1, n1), xv[32 + 4 * i], h);
            l = fmaf(fma_h(p0.y, s0, n0), xv[4 * i + 2], l); h = fmaf(fma_h(p1.y, s1, n1), xv[32 + 4 * i + 2], h);
            l = fmaf(fma_h(p2.x, s0, n0), xv[4 * i + 1], l); h = fmaf(fma_h(p3.x, s1, n1), xv[32 + 4 * i + 1], h);
            l = fmaf(fma_h(p2.y, s0, n0), xv[4 * i + 3], l); h = fmaf(fma_h(p3.y, s1, n1), xv[32 + 4 * i + 3], h);
            acc[c] = l; acc[c + 1] = h;
        }
        return (acc[0] + acc[2]) + (acc[1] + acc[3]);
    }
};
template <> struct Unit<QMM_Q6_K> {
    // Unit u = 4 sb + 2 h + lh: the 64 weights {128h + 32g + 16lh + i : g < 4,
    // i < 16} of super-block sb, which share one 16-byte slice of each ql half
    // and of qh.  Loads: A = ql[64h+16lh ..+16], B = ql[64h+32+16lh ..+16],
    // C = qh[32h+16lh ..+16], S = sc[8h ..+8], D = d.  Super-blocks are 210
    // bytes, so odd ones start 2 bytes off a dword: the loads are byte-
    // addressed (unaligned buffer loads), which keeps every window at its
    // own size and needs no realignment.
    static constexpr int NL = 4 + 4 + 4 + 2 + 1;
    struct Off { uint32_t a, c, s, d; int lh; };
    __device__ static Off lane_off(int u) {
        const int h = (u >> 1) & 1, lh = u & 1;
        const uint32_t base = 210u * (u >> 2);
        return {base + 64u * h + 16u * lh, base + 128u + 32u * h + 16u * lh, base + 192u + 8u * h, base + 208u, lh};
    }
    __device__ static void load(Rsrc rs, uint32_t row, const Off &o, uint32_t (&v)[NL]) {
        const u32x4_t a = __builtin_amdgcn_raw_buffer_load_b128(rs, o.a, row, 0);
        const u32x4_t b = __builtin_amdgcn_raw_buffer_load_b128(rs, o.a + 32u, row, 0);
        const u32x4_t c = __builtin_amdgcn_raw_buffer_load_b128(rs, o.c, row, 0);
        const u32x2_t sc = __builtin_amdgcn_raw_buffer_load_b64(rs, o.s, row, 0);
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
        v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
        v[8] = c.x; v[9] = c.y; v[10] = c.z; v[11] = c.w;
        v[12] = sc.x; v[13] = sc.y;
        v[14] = __builtin_amdgcn_raw_buffer_load_b16(rs, o.d, row, 0);
    }
    __device__ static int x4(int u, int i) {
        // unit u = 4b + 2h + lh covers x[256b + 128h + 32g + 16lh + j], g < 4, j < 16
        return 64 * (u >> 2) + 32 * ((u >> 1) & 1) + 8 * (i >> 2) + 4 * (u & 1) + (i & 3);
    }
    __device__ static float dot(const uint32_t (&v)[NL], const float (&xv)[64], const Off &o) {
        // code q = lo4 | hi2 << 4 per byte; (q - 32) 2^-24 as an exact f16 subnormal
        const half2_t b32 = as_h2(0x80208020u);  // -32 * 2^-24
        const float d = h2f(v[14]);
        float grp[4];
#pragma unroll
        for (int gp = 0; gp < 4; gp += 2) {  // two groups at a time: 8 independent chains
            half2_t w[2][4][2];  // [group][dword][bytes 0,2 | bytes 1,3]
#pragma unroll
            for (int k = 0; k < 2; k++) {
                const int g = gp + k;
#pragma unroll
                for (int t = 0; t < 4; t++) {
                    const uint32_t L = (g & 1) ? v[4 + t] : v[t];
                    const uint32_t C = v[8 + t];
                    const uint32_t hi = (g < 2 ? (C << (4 - 2 * g)) : (C >> (2 * g - 4))) & 0x30303030u;
                    const uint32_t q = ((g < 2 ? L : (L >> 4)) & 0x0F0F0F0Fu) | hi;
                    w[k][t][0] = as_h2(q & 0x00FF00FFu) + b32;
                    w[k][t][1] = as_h2(__builtin_amdgcn_perm(0u, q, 0x0C030C01u)) + b32;
                }
            }
            float s8[8];
#pragma unroll
            for (int k = 0; k < 2; k++)
#pragma unroll
                for (int t = 0; t < 4; t++) s8[4 * k + t] = fma_h(w[k][t][0].x, xv[16 * (gp + k) + 4 * t], 0.f);
#pragma unroll
            for (int k = 0; k < 2; k++)
#pragma unroll
                for (int t = 0; t < 4; t++) s8[4 * k + t] = fma_h(w[k][t][1].x, xv[16 * (gp + k) + 4 * t + 1], s8[4 * k + t]);
#pragma unroll
            for (int k = 0; k < 2; k++)
#pragma unroll
                for (int t = 0; t < 4; t++) s8[4 * k + t] = fma_h(w[k][t][0].y, xv[16 * (gp + k) + 4 * t + 2], s8[4 * k + t]);
#pragma unroll
            for (int k = 0; k < 2; k++)
#pragma unroll
                for (int t = 0; t < 4; t++) s8[4 * k + t] = fma_h(w[k][t][1].y, xv[16 * (gp + k) + 4 * t + 3], s8[4 * k + t]);
            grp[gp] = (s8[0] + s8[1]) + (s8[2] + s8[3]);
            grp[gp + 1] = (s8[4] + s8[5]) + (s8[6] + s8[7]);
        }
        float total = 0.f;
#pragma unroll
        for (int g = 0; g < 4; g++) {
            const uint32_t scw = (g < 2) ? v[12] : v[13];  // sc[8h .. 8h+4), sc[8h+4 .. 8h+8)
            const int sbyte = (int)__builtin_amdgcn_sbfe((int)scw, 16 * (g & 1) + 8 * o.lh, 8);  // sc[8h + 2g + lh]
            total = fmaf(d * 16777216.0f * (float)sbyte, grp[g], total);
        }
        return total;
    }
};

// ------------------------------------------------- activations in LDS ----
// Activations go through LDS laid out so that the 16 lanes of a read phase,
// each reading its own unit, hit distinct banks:
//   PAD    one float4 of padding after every 16 (17 float4s per 64 values):
//          a lane's 16 reads are one base address plus constant offsets
//          (whole-row wavefronts, 272 bytes per unit);
//   else   the float4 index XOR-swizzled within groups of 16 (256 bytes per
//          unit; per-read address arithmetic).
template <bool PAD>
__device__ __forceinline__ int xslot(int f) {
    if constexpr (PAD) return f + (f >> 4);
    else return (f & ~15) | ((f & 15) ^ ((f >> 4) & 15));
}
constexpr size_t xs_unit_bytes(bool pad) { return pad ? 272 : 256; }

// With PAD the offsets of a unit's float4s from its first one do not depend
// on the lane: every unit layout starts at a multiple of 16 or at 4 more, and
// its float4s lie at offsets o (< 28) with (first % 16) + (o % 16) < 16, so
// xslot(first + o) = xslot(first) + o + o / 16.
template <int DT, bool PAD>
__device__ __forceinline__ void x_from_lds(const floatx4 *xs, int u, float (&xv)[64]) {
    const int first = Unit<DT>::x4(u, 0);
#pragma unroll
    for (int i = 0; i < 16; i++) {
        const int o = Unit<DT>::x4(u, i) - first;
        const floatx4 v = PAD ? xs[xslot<true>(first) + o + (o >> 4)] : xs[xslot<false>(Unit<DT>::x4(u, i))];
        xv[4 * i] = v.x; xv[4 * i + 1] = v.y; xv[4 * i + 2] = v.z; xv[4 * i + 3] = v.w;
    }
}

// -------------------------------------------------- generic block dots ----
// Byte loads, any alignment: the same f32 arithmetic per block.
template <int DT>
__device__ float block_dot_generic(const uint8_t *blk, const float *x);

template <>
__device__ float block_dot_generic<QMM_Q4_0>(const uint8_t *p, const float *x) {
    const float d = h2f((uint32_t)p[0] | ((uint32_t)p[1] << 8));
    float slo = 0.f, shi = 0.f;
    for (int j = 0; j < 16; j++) {
        slo = fmaf((float)((int)(p[2 + j] & 15) - 8), x[j], slo);
        shi = fmaf((float)((int)(p[2 + j] >> 4) - 8), x[16 + j], shi);
    }
    return d * (slo + shi);
}

template <>
__device__ float block_dot_generic<QMM_Q4_1>(const uint8_t *p, const float *x) {
    const float d = h2f((uint32_t)p[0] | ((uint32_t)p[1] << 8));
    const float m = h2f((uint32_t)p[2] | ((uint32_t)p[3] << 8));
    float slo = 0.f, shi = 0.f;
    for (int j = 0; j < 16; j++) {
        slo = fmaf(fmaf(d, (float)(p[4 + j] & 15), m), x[j], slo);
        shi = fmaf(fmaf(d, (float)(p[4 + j] >> 4), m), x[16 + j], shi);
    }
    return slo + shi;
}

template <>
__device__ float block_dot_generic<QMM_Q8_0>(const uint8_t *p, const float *x) {
    const float d = h2f((uint32_t)p[0] | ((uint32_t)p[1] << 8));
    float s0 = 0.f, s1 = 0.f;
    for (int j = 0; j < 16; j++) {
        s0 = fmaf((float)(int8_t)p[2 + j], x[j], s0);
        s1 = fmaf((float)(int8_t)p[18 + j], x[16 + j], s1);
    }
    return d * (s0 + s1);
}

template <>
__device__ float block_dot_generic<QMM_Q4_K>(const uint8_t *p, const float *x) {
    const float d = h2f((uint32_t)p[0] | ((uint32_t)p[1] << 8));
    const float dmin = h2f((uint32_t)p[2] | ((uint32_t)p[3] << 8));
    uint32_t s[3];
    for (int i = 0; i < 3; i++)
        s[i] = (uint32_t)p[4 + 4 * i] | ((uint32_t)p[5 + 4 * i] << 8) | ((uint32_t)p[6 + 4 * i] << 16) |
               ((uint32_t)p[7 + 4 * i] << 24);
    float total = 0.f;
    for (int i = 0; i < 8; i++) {
        int sc, mn;
        q4k_scale_min(s[0], s[1], s[2], i, sc, mn);
        const float dsc = d * (float)sc, ndm = -(dmin * (float)mn);
        float s0 = 0.f, s1 = 0.f;
        for (int e = 0; e < 16; e++) {
            const uint8_t b0 = p[16 + 32 * (i >> 1) + e], b1 = p[16 + 32 * (i >> 1) + 16 + e];
            const float q0 = (float)((i & 1) ? (b0 >> 4) : (b0 & 15));
            const float q1 = (float)((i & 1) ? (b1 >> 4) : (b1 & 15));
            s0 = fmaf(fmaf(dsc, q0, ndm), x[32 * i + e], s0);
            s1 = fmaf(fmaf(dsc, q1, ndm), x[32 * i + 16 + e], s1);
        }
        total += s0 + s1;
    }
    return total;
}

template <>
__device__ float block_dot_generic<QMM_Q5_K>(const uint8_t *p, const float *x) {
    const float d = h2f((uint32_t)p[0] | ((uint32_t)p[1] << 8));
    const float dmin = h2f((uint32_t)p[2] | ((uint32_t)p[3] << 8));
    uint32_t s[3];
    for (int i = 0; i < 3; i++)
        s[i] = (uint32_t)p[4 + 4 * i] | ((uint32_t)p[5 + 4 * i] << 8) | ((uint32_t)p[6 + 4 * i] << 16) |
               ((uint32_t)p[7 + 4 * i] << 24);
    float total = 0.f;
    for (int i = 0; i < 8; i++) {
        int sc, mn;
        q4k_scale_min(s[0], s[1], s[2], i, sc, mn);
        const float dsc = d * (float)sc, ndm = -(dmin * (float)mn);
        float s0 = 0.f, s1 = 0.f;
        for (int e = 0; e < 16; e++) {
            const uint8_t b0 = p[48 + 32 * (i >> 1) + e], b1 = p[48 + 32 * (i >> 1) + 16 + e];
            const int h0 = (p[16 + e] >> i) & 1, h1 = (p[32 + e] >> i) & 1;
            const float q0 = (float)(((i & 1) ? (b0 >> 4) : (b0 & 15)) | (h0 << 4));
            const float q1 = (float)(((i & 1) ? (b1 >> 4) : (b1 & 15)) | (h1 << 4));
            s0 = fmaf(fmaf(dsc, q0, ndm), x[32 * i + e], s0);
            s1 = fmaf(fmaf(dsc, q1, ndm), x[32 * i + 16 + e], s1);
        }
        total += s0 + s1;
    }
    return total;
}

template <>
__device__ float block_dot_generic<QMM_Q6_K>(const uint8_t *p, const float *x) {
    const float d = h2f((uint32_t)p[208] | ((uint32_t)p[209] << 8));
    float total = 0.f;
    for (int s = 0; s < 16; s++) {  // 16 groups of 16 weights sharing one sub-scale
        const float dsc = d * (float)(int8_t)p[192 + s];
        float acc = 0.f;
        for (int i = 0; i < 16; i++) {
            const int j = 16 * s + i, h = j >> 7, g = (j & 127) >> 5, l = j & 31;
            const uint8_t lb = p[64 * h + 32 * (g & 1) + l];
            const int lo = (g < 2) ? (lb & 15) : (lb >> 4);
            const int hi = (p[128 + 32 * h + l] >> (2 * g)) & 3;
            acc = fmaf((float)((lo | (hi << 4)) - 32), x[j], acc);
        }
        total = fmaf(dsc, acc, total);
    }
    return total;
}

// Q8_0 quantization of four activations of a block whose other 28 sit in the
// seven neighbouring lanes (lanes 8j .. 8j+7 hold one block): the block's
// amax (a NaN never wins the comparison), d = amax/127, id = 1/d unless d is
// 0 or 1/d is not finite, codes = rint(v * id) clamped to [-128, 127] (NaN ->
// 0), packed little-endian; *d_out = d (the caller stores it rounded to f16).
// Every lane of the wavefront must call it.
//
// The lane maxima are combined across the 8 lanes with DPP moves inside the
// VALU (swap neighbours, swap pairs, mirror the half-row of 8: the same
// pattern as the first three steps of the wavefront sum), not with LDS
// permutes; a lane maximum is never NaN, so a plain max is exact there.  The
// clamp is done on the float before the conversion (NaN replaced first), so
// it compiles to selects, not branches.
template <int CTRL>
__device__ __forceinline__ float dpp_f(float v) {
    return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, 0xF, 0xF, true));
}
// the block maximum of |v| over the 8 lanes of the block
__device__ __forceinline__ float q8_block_amax(const floatx4 &v) {
    float amax = 0.f;
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const float a = fabsf(v[i]);
        amax = a > amax ? a : amax;
    }
    amax = fmaxf(amax, dpp_f<0xB1>(amax));   // quad_perm 1,0,3,2
    amax = fmaxf(amax, dpp_f<0x4E>(amax));   // quad_perm 2,3,0,1
    return fmaxf(amax, dpp_f<0x141>(amax));  // row_half_mirror
}
__device__ __forceinline__ void q8_scale(float amax, float &d, float &id) {
    d = amax / 127.0f;
    const float r = 1.0f / d;
    id = (d != 0.0f && __builtin_isfinite(r)) ? r : 0.0f;
}
__device__ __forceinline__ uint32_t q8_codes4(const floatx4 &v, float id) {
    uint32_t packed = 0;
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const float q = rintf(v[i] * id);
        const float qc = q != q ? 0.0f : fminf(fmaxf(q, -128.0f), 127.0f);
        packed |= ((uint32_t)(int)qc & 0xFFu) << (8 * i);
    }
    return packed;
}
__device__ __forceinline__ uint32_t q8_quant4(const floatx4 &v, float *d_out) {
    float d, id;
    q8_scale(q8_block_amax(v), d, id);
    *d_out = d;
    return q8_codes4(v, id);
}

}  // namespace qmm
