// qmm_attn.hip -- attention of a few new tokens over the paged cache (one
// decoded token, drafted tokens; include/qmm.h, qmm_attention), and the join of
// what several workgroups made of one row.
//
// Per row:  x_j = scale q . k_j,  out = sum_j 2^(x_j - m) v_j / sum_j 2^(x_j - m)
// (x in base 2, m its running maximum), one pass over the row's tokens.
//
// Bound by memory: every key and value is read once for all G query heads of its
// head and all new tokens (32/8 heads of 128, f16: one token over 131072 96 us and 5 for the join,
// 5.6 TB/s; 64 sequences of 1 to 8192 225 + 7 us, 5.4 TB/s); few rounds of a
// wavefront by latency (28 rows on a Q8_0 cache, 8 x 7 tokens to 4096: 33 + 5 us, a wavefront waits in 43 %
// of its cycles, vector ALU busy in 27; 513 tokens: 8.6 + 4.0).  The matrix cores do the products, because a row of f32
// FMAs would cost as many instructions per query head as there are bytes:
//   scores^T = K Q^T   v_mfma_f32_16x16x32_f16, A = 16 tokens' keys (a lane's 8
//                      values are 16 bytes of its token's key), B = 16 columns of
//                      queries
//   out^T   += V^T P^T A = 16 dims of the values (the pool holds them with the
//                      token inside: a lane's 8 tokens are 16 bytes), B = the
//                      probabilities, which the first product leaves in the lane
//                      that needs them: token 8 g + 4 t + i of a chunk of 32 is row
//                      4 g + i of product t, so lane (column, g) holds its 8 tokens
// f32 class: queries (under a power of two) and probabilities (times 2^15) are split
// in two f16 parts.  Up to 8 rows (G heads, one token) both parts sit in one
// tile's columns 0-7 and 8-15, at the price of one; more rows take two
// products.  Q8_0: a step of 32 dims is one block, so its product of codes is
// scaled by the token's key scale in f32; the value scale goes into the
// probability, under a running power of two as the maximum is.
//
// No LDS on the way in: a wavefront holds 32 tokens of keys and values in
// registers and asks for the next chunk's keys as soon as the scores are done, the
// next values after the second product.  The four wavefronts of a workgroup take
// every fourth chunk and join through LDS; workgroups that share a row write their
// sums and maxima to `work`, joined by a second launch.
#include "qmm_attn.hpp"

namespace qmm {

namespace {

constexpr int kWaves = 4, kChunk = 32, kLeast = 4;

template <int D, bool Q8> struct Regs;  // keys and values of a chunk
template <int D> struct Regs<D, false> {
    u32x4_t k[2][D / 32], v[D / 16];
};
template <int D> struct Regs<D, true> {
    u32x2_t k[2][D / 32], v[D / 16];
    half8 ks[D / 32], vs[D / 32];  // scales of tokens 8g .. 8g+7
};

// The pages of a lane's tokens of a chunk: the token whose key it loads is in group
// r / 4 of 8 (r = lane % 16), its values' and scores' tokens are group g = lane / 16.
// -1: the group has none; it reads page 0 and is masked.
struct Where {
    int k, v;
};

__device__ __forceinline__ Where where(const Pages &page_of, int k0) {
    const int lane = (int)threadIdx.x & 63;
    return Where{page_of(k0 + 8 * ((lane & 15) >> 2)), page_of(k0 + 8 * (lane >> 4))};
}

__device__ __forceinline__ const uint8_t *record_of(const AttnArgs &a, const uint8_t *pool, int page, int h, int64_t rec) {
    return pool + ((int64_t)(page < 0 ? 0 : page) * a.kv.heads + h) * rec;
}

template <int D, bool Q8>
__device__ __forceinline__ void load_keys(const AttnArgs &a, const Where &w, int h, int k0, int64_t rec, Regs<D, Q8> &x) {
    const int lane = (int)threadIdx.x & 63, r = lane & 15, g = lane >> 4, page = 1 << a.kv.page_shift;
    const uint8_t *p = record_of(a, a.kv.k, w.k, h, rec);
    const int slot = ((k0 + 8 * (r >> 2)) & (page - 1)) + (r & 3);
#pragma unroll
    for (int t = 0; t < 2; t++)
#pragma unroll
        for (int b = 0; b < D / 32; b++) {
            const int at = (slot + 4 * t) * D + 32 * b + 8 * g;
            if constexpr (Q8) x.k[t][b] = *reinterpret_cast<const u32x2_t *>(p + at);
            else x.k[t][b] = *reinterpret_cast<const u32x4_t *>(p + 2 * at);
        }
    if constexpr (Q8) {
        const uint8_t *ps = record_of(a, a.kv.k, w.v, h, rec) + page * D;
        const int s0 = (k0 + 8 * g) & (page - 1);
#pragma unroll
        for (int b = 0; b < D / 32; b++) x.ks[b] = *reinterpret_cast<const half8 *>(ps + 2 * (b * page + s0));
    }
}

template <int D, bool Q8>
__device__ __forceinline__ void load_values(const AttnArgs &a, const Where &w, int h, int k0, int64_t rec, Regs<D, Q8> &x) {
    const int lane = (int)threadIdx.x & 63, r = lane & 15, g = lane >> 4, page = 1 << a.kv.page_shift;
    const uint8_t *p = record_of(a, a.kv.v, w.v, h, rec);
    const int slot = (k0 + 8 * g) & (page - 1);
#pragma unroll
    for (int d = 0; d < D / 16; d++) {
        const int at = (16 * d + r) * page + slot;
        if constexpr (Q8) x.v[d] = *reinterpret_cast<const u32x2_t *>(p + at);
        else x.v[d] = *reinterpret_cast<const u32x4_t *>(p + 2 * at);
    }
    if constexpr (Q8) {
#pragma unroll
        for (int b = 0; b < D / 32; b++)
            x.vs[b] = *reinterpret_cast<const half8 *>(p + page * D + 2 * (b * page + slot));
    }
}

// MODE 0: up to 8 rows a workgroup, both parts in one column tile; 1, 2: one or
// two tiles of 16 rows, each part its own product.
template <int D, bool Q8, int MODE>
__global__ void __launch_bounds__(64 * kWaves, D > 128 ? 1 : MODE == 0 ? 3 : 2) attn_few_kernel(const AttnArgs a) {
    constexpr int NC = MODE == 0 ? 1 : MODE, RT = MODE == 0 ? 8 : 16 * MODE, NK = D / 32, ND = D / 16;
    constexpr bool STACK = MODE == 0;
    __shared__ __attribute__((aligned(16))) float lo_[kWaves][16][D + 4];
    __shared__ float2 lstat[kWaves][NC * 16];
    __shared__ half8 lq[STACK ? 1 : NC][STACK ? 1 : NK][2][STACK ? 1 : 64];
    __shared__ float lmul[STACK ? 1 : NC][16];
    AttnShare w;
    if (!attn_share<RT, kChunk>(a, kLeast, w)) return;
    const int lane = (int)threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int col = lane & 15, g = lane >> 4;
    const int64_t rec = kv_record(Q8 ? QMM_Q8_0 : QMM_F16, (int64_t)1 << a.kv.page_shift, D);

    const Pages page_of(a, w.s);
    int k0 = w.k0 + kChunk * wave;
    Regs<D, Q8> x;
    Where at{}, next{}, after{};
    if (k0 < w.k1) {
        at = where(page_of, k0);
        if constexpr (!STACK) next = where(page_of, k0 + kChunk * kWaves);
    }

    // the queries' two parts (one tile: in registers, every wavefront its own; more rows:
    // in LDS, made by a wavefront a tile), and what each of the lane's columns sees
    half8 qf[STACK ? NK : 1];
    float mul[NC];
    int lo[NC], hi[NC];
    int row[NC];
#pragma unroll
    for (int c = 0; c < NC; c++) {
        const int r = STACK ? (col & 7) : 16 * c + col;
        const bool on = r < w.nrows;
        row[c] = w.r0 + (on ? r : 0);
        attn_sees(a, w.nw, row[c] / a.G, lo[c], hi[c]);
        if (!on) lo[c] = hi[c] = 0;
    }
    auto queries = [&](int c, auto put) {
        const int t = row[c] / a.G, hq = w.h * a.G + (row[c] - t * a.G);
        const bool on = (STACK ? (col & 7) : 16 * c + col) < w.nrows;
        const float *q = a.Q + (int64_t)(w.nw.first + t) * a.q_stride + (int64_t)hq * D + 8 * g;
        floatx4 y[NK][2];
#pragma unroll
        for (int b = 0; b < NK; b++)
#pragma unroll
            for (int i = 0; i < 2; i++) y[b][i] = *reinterpret_cast<const floatx4 *>(q + 32 * b + 4 * i);
        // the first chunk is asked for before the queries are looked at
        if (c == 0 && k0 < w.k1) {
            load_keys<D, Q8>(a, at, w.h, k0, rec, x);
            load_values<D, Q8>(a, at, w.h, k0, rec, x);
        }
        float amax = 0.f;
#pragma unroll
        for (int b = 0; b < NK; b++)
#pragma unroll
            for (int i = 0; i < 8; i++) {
                if (!on) y[b][i / 4][i % 4] = 0.f;
                amax = fmaxf(amax, fabsf(y[b][i / 4][i % 4]));
            }
        const int e = row_exponent(fold32(fold16(amax, MaxOp()), MaxOp()));
#pragma unroll
        for (int b = 0; b < NK; b++) {
            half8 p, rest;
#pragma unroll
            for (int i = 0; i < 8; i++) {
                const float v = ldexpf(y[b][i / 4][i % 4], e);
                p[i] = (_Float16)v;
                rest[i] = (_Float16)(v - (float)p[i]);
            }
            put(b, p, rest);
        }
        return attn_mul(a, e);
    };
    if constexpr (STACK) {
        mul[0] = queries(0, [&](int b, half8 p, half8 rest) { qf[b] = col >= 8 ? rest : p; });
    } else {
#pragma unroll
        for (int c = 0; c < NC; c++) {
            if (wave == c) {
                const float m_ = queries(c, [&](int b, half8 p, half8 rest) {
                    lq[c][b][0][lane] = p;
                    lq[c][b][1][lane] = rest;
                });
                if (g == 0) lmul[c][col] = m_;
            }
        }
        if (wave != 0 && k0 < w.k1) {
            load_keys<D, Q8>(a, at, w.h, k0, rec, x);
            load_values<D, Q8>(a, at, w.h, k0, rec, x);
        }
        __syncthreads();
#pragma unroll
        for (int c = 0; c < NC; c++) mul[c] = lmul[c][col];
    }

    const float m1 = opaque_minus_one();
    floatx4 o[NC][ND];
    float m[NC], l[NC];
    int top[NC];  // Q8_0: biased exponent of the largest value scale
#pragma unroll
    for (int c = 0; c < NC; c++) {
        m[c] = -INFINITY;
        l[c] = 0.f;
        top[c] = 0;
#pragma unroll
        for (int d = 0; d < ND; d++) o[c][d] = floatx4{0.f, 0.f, 0.f, 0.f};
    }

    for (; k0 < w.k1; k0 += kChunk * kWaves) {
        const int kn = k0 + kChunk * kWaves;
        // The next chunk's pages.  With more than one tile's work in a chunk they are asked for a chunk
        // ahead, below, before the values: loads return in order, and the next keys' addresses would
        // wait for those values (8 x 7 tokens on Q8_0: 39.4 to 36.7 us; one token over 131072: 101 here, 113 so)
        if constexpr (STACK) {
            if (kn < w.k1) next = where(page_of, kn);
        }
        // scores: s[c][4 t + i] is token k0 + 8 g + 4 t + i of column c
        float s[NC][8];
        {
            floatx4 sum[2][NC];
#pragma unroll
            for (int t = 0; t < 2; t++)
#pragma unroll
                for (int c = 0; c < NC; c++) sum[t][c] = floatx4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int b = 0; b < NK; b++) {
                half8 kf[2];
#pragma unroll
                for (int t = 0; t < 2; t++) {
                    if constexpr (Q8) kf[t] = codes8(x.k[t][b]);
                    else kf[t] = __builtin_bit_cast(half8, x.k[t][b]);
                }
#pragma unroll
                for (int c = 0; c < NC; c++) {
                    half8 qh, ql;
                    if constexpr (STACK) {
                        qh = qf[b];
                    } else {
                        qh = lq[c][b][0][lane];
                        ql = lq[c][b][1][lane];
                    }
#pragma unroll
                    for (int t = 0; t < 2; t++) {
                        floatx4 z = Q8 ? floatx4{0.f, 0.f, 0.f, 0.f} : sum[t][c];
                        if constexpr (!STACK) z = __builtin_amdgcn_mfma_f32_16x16x32_f16(kf[t], ql, z, 0, 0, 0);
                        z = __builtin_amdgcn_mfma_f32_16x16x32_f16(kf[t], qh, z, 0, 0, 0);
                        if constexpr (Q8) {
#pragma unroll
                            for (int i = 0; i < 4; i++) sum[t][c][i] = fmaf(z[i], (float)x.ks[b][4 * t + i], sum[t][c][i]);
                        } else {
                            sum[t][c] = z;
                        }
                    }
                }
                if constexpr (Q8) __builtin_amdgcn_sched_barrier(0);
            }
#pragma unroll
            for (int c = 0; c < NC; c++)
#pragma unroll
                for (int t = 0; t < 2; t++)
#pragma unroll
                    for (int i = 0; i < 4; i++) {
                        float v = sum[t][c][i];
                        if constexpr (STACK)  // the other part's column: row_ror 8
                            v += __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), 0x128, 0xF, 0xF, true));
                        s[c][4 * t + i] = v * mul[c];
                    }
            if (a.cap > 0.f) {  // uniform
#pragma unroll
                for (int c = 0; c < NC; c++) cap_scores<8>(a, s[c]);
            }
        }
        if (kn < w.k1) {
            load_keys<D, Q8>(a, next, w.h, kn, rec, x);
            if constexpr (!STACK) after = where(page_of, kn + kChunk * kWaves);
        }

        const bool plain = k0 >= w.lo_all && k0 + kChunk <= w.hi_all && __ballot(at.v < 0) == 0;  // uniform
        if (!plain) {
#pragma unroll
            for (int c = 0; c < NC; c++)
#pragma unroll
                for (int j = 0; j < 8; j++) {
                    const int k = k0 + 8 * g + j;
                    if (at.v < 0 || k < lo[c] || k >= hi[c]) s[c][j] = -INFINITY;
                }
        }
        // what no row sees has no value, whatever the pool holds there.  What
        // some rows see and others do not must not reach the others through 0 *
        // infinity: such f16 values are taken out here and added by hand below
        bool odd = false;
        if (!plain) {
#pragma unroll
            for (int j = 0; j < 8; j++) {
                const int k = k0 + 8 * g + j;
                const bool any = at.v >= 0 && k >= w.lo_any && k < w.hi_any, all = at.v >= 0 && k >= w.lo_all && k < w.hi_all;
                if constexpr (Q8) {
#pragma unroll
                    for (int b = 0; b < NK; b++) {
                        const bool inf = !__builtin_isfinite((float)x.vs[b][j]);
                        odd |= inf && any && !all;
                        if (!any || (inf && !all)) x.vs[b][j] = (_Float16)0.f;
                    }
                } else {
                    const uint32_t sel = j & 1 ? 0xFFFF0000u : 0x0000FFFFu, exps = sel & 0x7C007C00u;
#pragma unroll
                    for (int d = 0; d < ND; d++) {
                        const uint32_t v = x.v[d][j / 2];
                        const bool inf = (v & exps) == exps;
                        odd |= inf && any && !all;
                        if (!any || (inf && !all)) x.v[d][j / 2] = v & ~sel;
                    }
                }
            }
        }
        // f16: probabilities are 2^15 times themselves, so that both parts of one below
        // 2^-14 keep their bits.  Q8_0: a probability times its token's value scale,
        // under the power of two that the scales the row has seen stay below, |scale| < 2^(top - 14)
        float grow[NC], unit[NC];
        if constexpr (Q8) {
            typedef unsigned short ushort2_t __attribute__((ext_vector_type(2)));
            ushort2_t es[4];  // tokens 2i and 2i + 1: the largest scale's bits
#pragma unroll
            for (int i = 0; i < 4; i++) {
                es[i] = ushort2_t{0, 0};
#pragma unroll
                for (int b = 0; b < NK; b++) {
                    const u32x4_t v = __builtin_bit_cast(u32x4_t, x.vs[b]);
                    const uint32_t u = v[i] & 0x7FFF7FFFu;
                    es[i] = __builtin_elementwise_max(es[i], __builtin_bit_cast(ushort2_t, u));
                }
            }
#pragma unroll
            for (int c = 0; c < NC; c++) {
                uint32_t e;
                if (plain) {
                    const ushort2_t m2 = __builtin_elementwise_max(__builtin_elementwise_max(es[0], es[1]), __builtin_elementwise_max(es[2], es[3]));
                    e = m2.x > m2.y ? m2.x : m2.y;
                } else {
                    e = 0;
#pragma unroll
                    for (int j = 0; j < 8; j++) {
                        const int k = k0 + 8 * g + j;
                        const uint32_t u = k >= lo[c] && k < hi[c] ? es[j / 2][j & 1] : 0u;
                        e = u > e ? u : e;
                    }
                }
                const int now = (int)fold32(fold16((float)(e >> 10), MaxOp()), MaxOp());
                const int up = now > top[c] ? now : top[c];
                grow[c] = ldexpf(1.f, top[c] - up);
                top[c] = up;
                unit[c] = ldexpf(1.f, 29 - up);
            }
        } else {
#pragma unroll
            for (int c = 0; c < NC; c++) grow[c] = 1.f;
        }
#pragma unroll
        for (int c = 0; c < NC; c++) {
            float mx = s[c][0];
#pragma unroll
            for (int j = 1; j < 8; j++) mx = fmaxf(mx, s[c][j]);
            mx = fmaxf(m[c], fold32(fold16(mx, MaxOp()), MaxOp()));
            const float ref = mx == -INFINITY ? 0.f : mx - (Q8 ? 0.f : 15.f), was = m[c] - (Q8 ? 0.f : 15.f);
            const float alpha = __builtin_amdgcn_exp2f(was - ref);
            m[c] = mx;
            float ps = 0.f;
#pragma unroll
            for (int j = 0; j < 8; j++) {
                s[c][j] = __builtin_amdgcn_exp2f(s[c][j] - ref);
                ps += s[c][j];
                if constexpr (Q8) s[c][j] *= unit[c];
            }
            l[c] = fmaf(l[c], alpha, ps);
            const float f = alpha * grow[c];
            if (__ballot(f != 1.f)) {
#pragma unroll
                for (int d = 0; d < ND; d++)
#pragma unroll
                    for (int i = 0; i < 4; i++) o[c][d][i] *= f;
            }
        }
        half8 ph[NC], pl[NC];
        auto parts = [&](int b) {
#pragma unroll
            for (int c = 0; c < NC; c++)
#pragma unroll
                for (int j = 0; j < 8; j += 2) {
                    half2_t h, r;
                    if constexpr (Q8) split2(s[c][j] * (float)x.vs[b][j], s[c][j + 1] * (float)x.vs[b][j + 1], m1, h, r);
                    else split2(s[c][j], s[c][j + 1], m1, h, r);
                    if (STACK) h = col >= 8 ? r : h;
                    ph[c][j] = h.x, ph[c][j + 1] = h.y;
                    pl[c][j] = r.x, pl[c][j + 1] = r.y;
                }
        };
        if constexpr (!Q8) parts(0);
#pragma unroll
        for (int b = 0; b < NK; b++) {
            half8 v0, v1;
            if constexpr (Q8) {
                v0 = codes8(x.v[2 * b]);
                v1 = codes8(x.v[2 * b + 1]);
                parts(b);
            } else {
                v0 = __builtin_bit_cast(half8, x.v[2 * b]);
                v1 = __builtin_bit_cast(half8, x.v[2 * b + 1]);
            }
#pragma unroll
            for (int c = 0; c < NC; c++) {
                if constexpr (!STACK) {
                    o[c][2 * b] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v0, pl[c], o[c][2 * b], 0, 0, 0);
                    o[c][2 * b + 1] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v1, pl[c], o[c][2 * b + 1], 0, 0, 0);
                }
                o[c][2 * b] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v0, ph[c], o[c][2 * b], 0, 0, 0);
                o[c][2 * b + 1] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v1, ph[c], o[c][2 * b + 1], 0, 0, 0);
            }
            // the blocks' conversions one after the other: all at once they spill
            if constexpr (Q8) __builtin_amdgcn_sched_barrier(0);
        }
        if (__ballot(odd)) {  // uniform; rare: an infinity or NaN that only some rows see
            for (int j = 0; j < kChunk; j++) {
                const int k = k0 + j, pg = page_of(k);
                if (pg < 0 || (k >= w.lo_all && k < w.hi_all)) continue;
                const int page = 1 << a.kv.page_shift, slot = k & (page - 1);
                const uint8_t *p = record_of(a, a.kv.v, pg, w.h, rec);
#pragma unroll
                for (int d = 0; d < ND; d++)
#pragma unroll
                    for (int i = 0; i < 4; i++) {
                        // addresses made here each time, not kept in registers through the main loop
                        int dim = 16 * d + 4 * g + i;
                        asm volatile("" : "+v"(dim));
                        float y;
                        if constexpr (Q8)
                            y = (float)reinterpret_cast<const int8_t *>(p)[dim * page + slot] *
                                (float)reinterpret_cast<const _Float16 *>(p + page * D)[(dim >> 5) * page + slot];
                        else
                            y = (float)reinterpret_cast<const _Float16 *>(p)[dim * page + slot];
                        if (__builtin_isfinite(y)) continue;
#pragma unroll
                        for (int c = 0; c < NC; c++)
                            if (k >= lo[c] && k < hi[c]) o[c][d][i] += y;
                    }
            }
        }
        at = next;
        if constexpr (!STACK) next = after;
        if (kn < w.k1) load_values<D, Q8>(a, at, w.h, kn, rec, x);
    }

    // join the wavefronts
#pragma unroll
    for (int c = 0; c < NC; c++) {
        l[c] = fold32(fold16(l[c], SumOp()), SumOp());
        if (l[c] != l[c]) m[c] = INFINITY;  // a NaN score is no maximum, but its row is not one that saw nothing
        if constexpr (!Q8) m[c] -= 15.f;  // probabilities and sums are 2^15 times theirs
        if (g == 0) lstat[wave][16 * c + col] = make_float2(m[c], l[c]);
    }
#pragma unroll
    for (int c = 0; c < NC; c++) {
        const float down = Q8 ? ldexpf(1.f, top[c] - 29) : 1.f;
        __syncthreads();
        float M = -INFINITY;
#pragma unroll
        for (int v = 0; v < kWaves; v++) M = fmaxf(M, lstat[v][16 * c + col].x);
        const float f = m[c] == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(m[c] - M) * down;
#pragma unroll
        for (int d = 0; d < ND; d++) {
            floatx4 y = o[c][d];
#pragma unroll
            for (int i = 0; i < 4; i++) y[i] = f == 0.f ? 0.f : y[i] * f;
            *reinterpret_cast<floatx4 *>(&lo_[wave][col][16 * d + 4 * g]) = y;
        }
        __syncthreads();
        const int rows = w.nrows - 16 * c < (STACK ? 8 : 16) ? w.nrows - 16 * c : (STACK ? 8 : 16);
        for (int e = (int)threadIdx.x; e < rows * (D / 4); e += 64 * kWaves) {
            const int r = e / (D / 4), d = 4 * (e - r * (D / 4));
            floatx4 y{};
            float Mr = -INFINITY, L = 0.f;
#pragma unroll
            for (int v = 0; v < kWaves; v++) Mr = fmaxf(Mr, lstat[v][16 * c + r].x);
#pragma unroll
            for (int v = 0; v < kWaves; v++) {
                const float2 st = lstat[v][16 * c + r];
                if (st.x != -INFINITY) L = fmaf(st.y, __builtin_amdgcn_exp2f(st.x - Mr), L);
                floatx4 z = *reinterpret_cast<const floatx4 *>(&lo_[v][r][d]);
                if constexpr (STACK) z += *reinterpret_cast<const floatx4 *>(&lo_[v][r + 8][d]);
                y += z;
            }
            const int row = w.r0 + 16 * c + r, t = row / a.G, hq = w.h * a.G + (row - t * a.G);
            const int64_t rh = (int64_t)(w.nw.first + t) * a.Hq + hq;
            if (a.splits == 1) {
                const float inv = L == 0.f ? 0.f : 1.f / L;
#pragma unroll
                for (int i = 0; i < 4; i++) y[i] *= inv;
                *reinterpret_cast<floatx4 *>(a.out + rh * D + d) = y;
            } else {
                const int64_t at_ = rh * a.splits + w.split;
                if (Mr != -INFINITY) *reinterpret_cast<floatx4 *>(a.part + at_ * D + d) = y;
                if (d == 0) a.stat[at_] = make_float2(Mr, L);
            }
        }
    }
}

// Rows that several workgroups share: out = sum_s 2^(m_s - M) part_s / sum_s
// 2^(m_s - M) l_s.  W wavefronts a row take every W-th split.
template <int D, int W>
__global__ void __launch_bounds__(256) attn_join_kernel(const AttnArgs a) {
    constexpr int NV = (D + 63) / 64, NB = 2;  // at most 64 NB splits
    __shared__ float acc[4][D];
    const int lane = (int)threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int64_t rh = (a.block0 + blockIdx.x) * (4 / W) + (W == 4 ? 0 : wave);
    if (rh >= (int64_t)a.kv.rows * a.Hq) return;  // W 1: whole wavefronts, no barrier follows
    // the statistics are asked for before the row is known to be one; a lane a split
    float2 st[NB];
#pragma unroll
    for (int b = 0; b < NB; b++)
        st[b] = 64 * b + lane < a.splits ? a.stat[rh * a.splits + 64 * b + lane] : make_float2(-INFINITY, 0.f);
    const int n = (int)(rh / a.Hq);
    const int s = kv_row_seq(a.kv, n);
    if (s < 0) return;
    const KvNew nw = kv_new(a.kv, s);
    if (n - nw.first >= nw.count) return;
    float M = fmaxf(st[0].x, st[1].x);
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) M = fmaxf(M, __shfl_xor(M, o, 64));
    float f[NB], L = 0.f;
#pragma unroll
    for (int b = 0; b < NB; b++) {
        f[b] = st[b].x == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(st[b].x - M);
        L += f[b] == 0.f ? 0.f : st[b].y * f[b];
    }
    L = wave_sum(L);
    const float *part = a.part + rh * a.splits * D;
    float y[NV] = {};
#pragma unroll
    for (int b = 0; b < NB; b++) {
        const int i1 = a.splits - 64 * b < 64 ? a.splits - 64 * b : 64;
#pragma unroll 8
        for (int i = W == 4 ? wave : 0; i < i1; i += W) {
            const float fi = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, f[b]), i));
#pragma unroll
            for (int v = 0; v < NV; v++) {
                // a split that saw nothing wrote nothing: what lies there may be NaN
                const float p = 64 * v + lane < D ? part[(int64_t)(64 * b + i) * D + 64 * v + lane] : 0.f;
                y[v] += fi == 0.f ? 0.f : p * fi;
            }
        }
    }
    if constexpr (W == 4) {
#pragma unroll
        for (int v = 0; v < NV; v++)
            if (64 * v + lane < D) acc[wave][64 * v + lane] = y[v];
        __syncthreads();
        if (wave != 0) return;
#pragma unroll
        for (int v = 0; v < NV; v++)
            if (64 * v + lane < D) y[v] = (acc[0][64 * v + lane] + acc[1][64 * v + lane]) + (acc[2][64 * v + lane] + acc[3][64 * v + lane]);
    }
    const float inv = L == 0.f ? 0.f : 1.f / L;
#pragma unroll
    for (int v = 0; v < NV; v++)
        if (64 * v + lane < D) a.out[rh * D + 64 * v + lane] = y[v] * inv;
}

// How a call is shared out: rows of a tile, row tiles of a sequence and head, splits of the tokens;
// by sizes that the host knows, so that a captured call keeps it.  Measured with 32 query and 8
// key-value heads of 128 (f16 unless said otherwise; a captured graph over inputs that rotate):
//   form    rows of a key-value head (new tokens x G): up to 16 in one tile of 16 26.5 us (the form
//           for many rows 31.8), 32 in two 30.0 (33.3), Q8_0 30.8 (38.9); 8 sequences of 2048.  128: the
//           form for many rows 46.5, four passes of this one 60.8.  48 and 64 rows in two
//           passes would be 3 % (Q8_0 11 %) faster there, where the second reads its keys
//           from the caches, and read them twice from memory in a larger batch
//   splits  few workgroups: enough splits that there are 256, of at least 128 tokens (513
//           tokens: 12.1 us; of 256 tokens 14.4); many: up to 4096 workgroups of at least 512 tokens
//           for the balance, at most 32 splits of a row (64 sequences of 1 to 8192: 232 us,
//           2048 workgroups 237, 512 without splits 279; 131072 tokens in 32 splits 101, 64
//           104, 128 111)
//   many rows: 512 workgroups, two a CU (512 tokens over 8192: 140 us; 256 180, 1024 167)
struct Plan {
    int mode;  // 0, 1, 2: attn_few_kernel; 3: the form for many rows
    int tiles, splits;
    int64_t blocks;
};

Plan plan_of(const qmm_kv_cache &c, const qmm_kv_batch &b, int64_t q_heads) {
    const int64_t G = q_heads / c.heads, rows = b.max_new * G, units = b.seqs * c.heads;
    Plan p;
    p.mode = rows >= tuning_lever("QMM_ATTN_PROMPT_FROM", 33) ? 3 : rows <= 8 ? 0 : rows <= 16 ? 1 : 2;
    const int64_t rt = p.mode == 0 ? 8 : p.mode == 3 ? kPromptRows : 16 * p.mode;
    p.tiles = (int)((rows + rt - 1) / rt);
    const int64_t groups = units * p.tiles, tokens = b.max_pages * c.page;
    // so many splits that there are `total` workgroups, of at least `least` tokens each
    auto share = [&](int64_t total, int64_t least) {
        const int64_t want = (total + groups - 1) / groups, most = (tokens + least - 1) / least;
        return want < most ? want : most;
    };
    int64_t s;
    if (p.mode == 3) {
        s = share(tuning_lever("QMM_ATTN_PROMPT_GROUPS", 512), tuning_lever("QMM_ATTN_PROMPT_LEAST", 256));
    } else {
        const int64_t wide = share(tuning_lever("QMM_ATTN_FILL", 256), tuning_lever("QMM_ATTN_FILL_LEAST", 128)),
                      even = share(tuning_lever("QMM_ATTN_GROUPS", 4096), tuning_lever("QMM_ATTN_LEAST", 512));
        const int64_t most = tuning_lever("QMM_ATTN_SPLITS", 32);  // for the balance: each costs the join a read
        s = even < most ? even : most;
        s = wide > s ? wide : s;
    }
    const int64_t cap = 128;  // what the join holds
    p.splits = (int)(s < 1 ? 1 : s > cap ? cap : s);
    p.blocks = units * p.tiles * p.splits;
    return p;
}

constexpr int64_t kBlocks = int64_t(1) << 23;  // of a launch: fewer than 2^32 threads

template <int D, bool Q8>
hipError_t launch_few(AttnArgs a, const Plan &p, hipStream_t st) {
    for (int64_t b = 0; b < p.blocks; b += kBlocks) {
        a.block0 = b;
        const dim3 grid((unsigned)(p.blocks - b < kBlocks ? p.blocks - b : kBlocks)), block(64 * kWaves);
        if (p.mode == 0) hipLaunchKernelGGL((attn_few_kernel<D, Q8, 0>), grid, block, 0, st, a);
        else if (p.mode == 1) hipLaunchKernelGGL((attn_few_kernel<D, Q8, 1>), grid, block, 0, st, a);
        else hipLaunchKernelGGL((attn_few_kernel<D, Q8, 2>), grid, block, 0, st, a);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

template <int D>
hipError_t launch_d(AttnArgs a, int dtype, const Plan &p, hipStream_t st) {
    const hipError_t e = p.mode == 3           ? launch_attn_prompt(a, dtype, D, p.blocks, st)
                         : dtype == QMM_Q8_0 ? launch_few<D, true>(a, p, st)
                                             : launch_few<D, false>(a, p, st);
    if (e != hipSuccess || p.splits == 1) return e;
    const int64_t rh = (int64_t)a.kv.rows * a.Hq;
    const bool wide = p.splits > 8;
    const int64_t blocks = wide ? rh : (rh + 3) / 4;
    for (int64_t b = 0; b < blocks; b += kBlocks) {
        a.block0 = b;
        const dim3 grid((unsigned)(blocks - b < kBlocks ? blocks - b : kBlocks));
        if (wide) hipLaunchKernelGGL((attn_join_kernel<D, 4>), grid, dim3(256), 0, st, a);
        else hipLaunchKernelGGL((attn_join_kernel<D, 1>), grid, dim3(256), 0, st, a);
        const hipError_t e2 = hipGetLastError();
        if (e2 != hipSuccess) return e2;
    }
    return hipSuccess;
}

// A positive value as f32, cut to the largest.
float f32_of(double v) { return v < FLT_MAX ? (float)v : FLT_MAX; }

}  // namespace

int64_t attention_work_bytes(const qmm_kv_cache &cache, const qmm_kv_batch &batch, int64_t q_heads) {
    const Plan p = plan_of(cache, batch, q_heads);
    return p.splits == 1 ? 0 : batch.rows * q_heads * p.splits * (4 * (int64_t)cache.dim + 8);
}

hipError_t launch_attention(const qmm_kv_cache &cache, const qmm_kv_batch &batch, const float *Q, int64_t q_stride,
                            int64_t q_heads, double scale, bool causal, int64_t window, double softcap, float *out,
                            void *work, hipStream_t st) {
    const Plan p = plan_of(cache, batch, q_heads);
    AttnArgs a{};
    a.Q = Q;
    a.out = out;
    a.part = (float *)work;
    a.stat = (float2 *)((char *)work + batch.rows * q_heads * p.splits * 4 * (int64_t)cache.dim);
    a.q_stride = q_stride;
    a.window = window;
    constexpr double log2e = 1.44269504088896340736;
    a.mul = (float)frexp(scale * log2e, &a.mul_exp);
    if (softcap > 0.0) {
        const double cap = softcap * log2e;
        a.cap = fmaxf(f32_of(cap), FLT_TRUE_MIN);  // one that rounds to 0 is still a cap
        a.cap_inv = f32_of(0.60196578275345014 / cap);  // the unit that makes P's leading coefficient 1
        a.cap_from = f32_of(0.5 * cap);
        a.cap_rate = f32_of(2.0 / softcap);  // e^(2t/c) = 2^(t rate)
    }
    a.Hq = (int)q_heads;
    a.G = (int)(q_heads / cache.heads);
    a.splits = p.splits;
    a.tiles = p.tiles;
    a.causal = causal;
    a.kv = kv_args(cache, batch);
    switch (cache.dim) {
    case 64: return launch_d<64>(a, cache.dtype, p, st);
    case 96: return launch_d<96>(a, cache.dtype, p, st);
    case 128: return launch_d<128>(a, cache.dtype, p, st);
    case 192: return launch_d<192>(a, cache.dtype, p, st);
    case 256: return launch_d<256>(a, cache.dtype, p, st);
    default: return hipErrorInvalidValue;
    }
}

}  // namespace qmm
