// qmm_attn_prompt.hip -- attention of many new tokens over the paged cache (a
// prompt, a chunk of one, long drafts; include/qmm.h, qmm_attention).
//
// A workgroup takes 128 rows (new tokens x the G query heads of one key-value
// head, so that they share every key) and 64 tokens of the cache at a time; a
// wavefront has 32 rows as the columns of v_mfma_f32_32x32x16_f16:
//   scores^T = K Q^T   A = 32 tokens' keys, B = the queries (registers)
//   out^T   += V^T P^T A = 32 dims of the values, B = the probabilities, which
//                      stay in the lane that made them: row r of the first
//                      product is token r with bits 2 and 3 exchanged, so a lane's
//                      16 scores are two runs of 8 neighbouring tokens
// f32 class: queries and probabilities in two f16 parts, two steps for one.
// Q8_0: codes times (both parts of) the queries, one block's product scaled by
// the token's key scale in f32; values times 2^7 as hi + lo, both f16 and exact together (a code
// times a scale has 18 bits and is 2^-24 at least), three steps for one: hi takes both parts of the
// probabilities, lo (2^-11 of the value or less, and 0 where the value is below 2^-20) their first.  Times
// 2^7, because the matrix cores align a product as if a factor below 2^-14 were as large as that.
// Values under scales from 4 on would pass f16 so: they go through products of their own.
//
// Bound by the matrix cores and by what a tile waits for: the products of a wavefront and tile take 2048
// cycles of a SIMD at D = 128, its softmax about 1100 of the vector ALU; two wavefronts a SIMD, and two
// halves of a tile in each, let one's softmax run under the other's products.  512 tokens over 8192,
// 32/8 heads of 128 f16: 133 us, 147 (median of 60) as the clock comes down (1000 and 905 TFLOP/s of f16 steps, where the
// library's plain product reaches 1160 to 1180; matrix cores busy in 48 % of the cycles, vector ALU in 36) and 11
// for the join.  At D = 64, half the products for the same softmax, neither is half busy (ragged Q8_0
// prompts: 23 and 43 %, a wavefront waits in 38 % of its cycles); 512 over 4096 51 us, Q8_0 65.  Keys and
// values go through registers to LDS (rows padded by 16 bytes: eight neighbouring rows
// then start in eight different groups of four banks), the next tile's loads under
// way during the products.
//
// The running reference of the exponentials moves only when a row's maximum
// passes it by 2^8: probabilities are up to 2^15 instead of 1, which both f16
// parts hold, and the outputs are rescaled once or twice a row instead of every tile.
#include "qmm_attn.hpp"

namespace qmm {

namespace {

constexpr int CH = kPromptChunk, RT = kPromptRows;
constexpr int AHEAD = 2;  // steps that a read from LDS is ahead of its products (3: 8 % slower, the registers spill)

// One tile on its way from memory to LDS.  Wavefront w brings the keys of the
// tile's w-th run of 16 tokens (neighbours in their page: one piece of memory, from a
// uniform address) and D/4 dims of all 64 tokens' values.
template <int D, bool Q8> struct Stage;
template <int D> struct Stage<D, false> {
    u32x4_t k[D / 32], v[D / 32];
};
template <int D> struct Stage<D, true> {
    // the wavefront's 8 dims of step i lie in one block: block (w D/4 + 8 i) / 32
    static constexpr int NB = D == 64 || D == 128 ? 1 : D == 256 ? 2 : D / 32;
    static __device__ constexpr int at(int i) { return NB == 1 ? 0 : NB == 2 ? i / 4 : i; }
    u32x2_t k[D / 32], v[D / 32];
    half8 vs[NB];
    u32x2_t ks;  // the thread's 4 tokens' scales of one block
};

template <int D, bool Q8> struct Tile {  // in LDS
    static constexpr int KP = D + 8, VP = CH + 8;
    _Float16 k[CH][KP];
    _Float16 v[Q8 ? 2 : 1][D][VP];
    _Float16 ks[Q8 ? D / 32 : 1][CH];
    int odd[4];  // per wavefront
    int large;   // the last tile with values under large scales
    // the queries' second parts of the first QL steps, a wavefront's own, where the registers cannot
    // hold them and this does (16 query heads of 256, 512 tokens over 4096: f16 131 us, 160 with 133
    // registers spilled; Q8_0 222, with 8 steps 8 % more, with none 40 %)
    static constexpr int QL = D != 256 ? 0 : Q8 ? 12 : 16;
    half8 ql[QL ? 4 : 1][QL ? QL : 1][QL ? 64 : 1];
};

// Token t of a tile <-> row of the first product: bits 2 and 3 exchanged.
__device__ __forceinline__ int swap23(int t) { return (t & ~12) | ((t & 4) << 1) | ((t & 8) >> 1); }

constexpr uint32_t kLargeScale = 0x4400, kInfScale = 0x7C00;  // f16 bits: 4, from where 2^7 of a value may pass 65504

// A value scale whose codes go through large_values.
__device__ __forceinline__ bool is_large(_Float16 scale) {
    const uint32_t u = __builtin_bit_cast(unsigned short, scale) & 0x7FFFu;
    return u >= kLargeScale && u < kInfScale;
}

// A token's distance from the tile's first, cut to what the tile can tell apart.
__device__ __forceinline__ int within(int x) { return x < 0 ? 0 : x > CH ? CH : x; }

template <int D, bool Q8>
__global__ void __launch_bounds__(256, D <= 128 ? 2 : 1) attn_prompt_kernel(const AttnArgs a) {
    constexpr int NS = D / 32, NK = D / 16, ND = D / 32;
    extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
    Tile<D, Q8> &T = *reinterpret_cast<Tile<D, Q8> *>(lds);
    AttnShare w;
    if (!attn_share<RT, CH>(a, 2, w)) return;
    const int tid = (int)threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int col = lane & 31, hh = lane >> 5;
    const int page = 1 << a.kv.page_shift;
    const int64_t rec = kv_record(Q8 ? QMM_Q8_0 : QMM_F16, page, D);
    const int r = 32 * wave + col;
    const bool on = r < w.nrows, wave_on = 32 * wave < w.nrows;
    const int row = w.r0 + (on ? r : 0), t = row / a.G, hq = w.h * a.G + (row - t * a.G);
    int lo, hi;
    attn_sees(a, w.nw, t, lo, hi);
    if (!on) lo = hi = 0;

    constexpr int QL = Tile<D, Q8>::QL;
    half8 qh[NK], ql[QL < NK ? NK - QL : 1];
    float mul;
    {
        const float *q = a.Q + (int64_t)(w.nw.first + t) * a.q_stride + (int64_t)hq * D + 8 * hh;
        float amax = 0.f;
        floatx4 x[NK][2];
#pragma unroll
        for (int b = 0; b < NK; b++)
#pragma unroll
            for (int i = 0; i < 2; i++) {
                x[b][i] = *reinterpret_cast<const floatx4 *>(q + 16 * b + 4 * i);
#pragma unroll
                for (int j = 0; j < 4; j++) {
                    if (!on) x[b][i][j] = 0.f;
                    amax = fmaxf(amax, fabsf(x[b][i][j]));
                }
            }
        amax = fold32(amax, MaxOp());
        const int e = row_exponent(amax);
        mul = attn_mul(a, e);
        // a negative scale goes into the queries, so that the largest product is the largest score
        const bool neg = mul < 0.f;
        mul = fmaxf(fabsf(mul), 0x1p-126f);  // above 0: a masked -inf stays one
#pragma unroll
        for (int b = 0; b < NK; b++) {
            half8 rest;
#pragma unroll
            for (int i = 0; i < 8; i++) {
                const float s = x[b][i / 4][i % 4], v = ldexpf(neg ? -s : s, e);
                const _Float16 p = (_Float16)v;
                qh[b][i] = p;
                rest[i] = (_Float16)(v - (float)p);
            }
            if (b < QL) T.ql[wave][b][lane] = rest;
            else ql[b - QL] = rest;
        }
    }
    floatx16 o[ND];
#pragma unroll
    for (int d = 0; d < ND; d++)
#pragma unroll
        for (int i = 0; i < 16; i++) o[d][i] = 0.f;
    float base = -INFINITY, l = 0.f;
    const float m1 = opaque_minus_one();

    Stage<D, Q8> st;
    int good = 0;  // which of the tile's four runs of 16 tokens have a page
    const int g = lane & 7, d0 = wave * (D / 4) + (lane >> 3);  // the values' tokens 8g .. 8g+7 and dims d0 + 8i
    const Pages page_of(a, w.s);
    int pg = page_of(w.k0 + 16 * (lane & 3));  // lane r % 4: the page of the next tile's run r
    auto load = [&](int k0) {
        good = (int)__ballot(pg >= 0) & 15;
        const int at = pg < 0 ? 0 : pg;  // masked
        const uint8_t *kr = a.kv.k + ((int64_t)__builtin_amdgcn_readlane(at, wave) * a.kv.heads + w.h) * rec;
        const int pv = __shfl(at, g >> 1, 64);
        const uint8_t *vr = a.kv.v + ((int64_t)pv * a.kv.heads + w.h) * rec;
        const int kslot = (k0 + 16 * wave) & (page - 1);
#pragma unroll
        for (int i = 0; i < NS; i++) {
            if constexpr (Q8) st.k[i] = *reinterpret_cast<const u32x2_t *>(kr + kslot * D + 8 * lane + 512 * i);
            else st.k[i] = *reinterpret_cast<const u32x4_t *>(kr + 2 * kslot * D + 16 * lane + 1024 * i);
        }
        if constexpr (Q8) {
            if (tid < 16 * NS) {
                const int b = tid >> 4, key = 4 * (tid & 15);
                const uint8_t *p = a.kv.k + ((int64_t)__shfl(at, key >> 4, 64) * a.kv.heads + w.h) * rec + page * D;
                st.ks = *reinterpret_cast<const u32x2_t *>(p + 2 * (b * page + ((k0 + key) & (page - 1))));
            }
        }
        const int vslot = (k0 + 8 * g) & (page - 1);
#pragma unroll
        for (int i = 0; i < NS; i++) {
            const int at = (d0 + 8 * i) * page + vslot;
            if constexpr (Q8) st.v[i] = *reinterpret_cast<const u32x2_t *>(vr + at);
            else st.v[i] = *reinterpret_cast<const u32x4_t *>(vr + 2 * at);
        }
        if constexpr (Q8) {
#pragma unroll
            for (int i = 0; i < NS; i++)
                if (i == 0 || st.at(i) != st.at(i - 1))
                    st.vs[st.at(i)] = *reinterpret_cast<const half8 *>(
                        vr + page * D + 2 * (((wave * (D / 4) + 8 * i) >> 5) * page + vslot));
        }
        pg = page_of(k0 + CH + 16 * (lane & 3));
    };
    // the tile to LDS; `plain`: every row sees all of it.  What no row sees has no
    // value, whatever the pool holds; infinities and NaN that only some rows see are
    // taken out (T.odd) and added by hand
    auto store = [&](int k0, bool plain) {
#pragma unroll
        for (int i = 0; i < NS; i++) {
            const int e = lane + 64 * i, key = e / (D / 8), c = e - key * (D / 8);
            half8 x;
            if constexpr (Q8) x = codes8(st.k[i]);
            else x = __builtin_bit_cast(half8, st.k[i]);
            *reinterpret_cast<half8 *>(&T.k[16 * wave + swap23(key)][8 * c]) = x;
        }
        if constexpr (Q8) {
            if (tid < 16 * NS) *reinterpret_cast<u32x2_t *>(&T.ks[tid >> 4][4 * (tid & 15)]) = st.ks;
        }
        bool odd = false, large = false;
        if constexpr (Q8) {
            // values under large scales are taken out here, like those that no row sees, and come from large_values
            // (a negative scale, which no quantizer makes, is looked at too)
            typedef unsigned short ushort2_t __attribute__((ext_vector_type(2)));
            ushort2_t most{0, 0};
#pragma unroll
            for (int b = 0; b < Stage<D, Q8>::NB; b++) {
                const u32x4_t v = __builtin_bit_cast(u32x4_t, st.vs[b]);
#pragma unroll
                for (int j = 0; j < 4; j++) {
                    const uint32_t u = v[j];
                    most = __builtin_elementwise_max(most, __builtin_bit_cast(ushort2_t, u));
                }
            }
            if (__ballot(most.x >= kLargeScale || most.y >= kLargeScale)) {  // rare
#pragma unroll
                for (int b = 0; b < Stage<D, Q8>::NB; b++)
#pragma unroll
                    for (int j = 0; j < 8; j++) {
                        if (!is_large(st.vs[b][j])) continue;
                        large = true;
                        st.vs[b][j] = (_Float16)0.f;
                    }
            }
        }
#pragma unroll
        for (int i = 0; i < NS; i++) {
            const int d = d0 + 8 * i;
            half8 x, y;
            if constexpr (Q8) {
                // 2^7 v = x + y exactly: v is a multiple of its scale's last bit, 2^18 of them at most
                const half8 cd = codes8(st.v[i]), sc = st.vs[st.at(i)] * (_Float16)128.f;
#pragma unroll
                for (int j = 0; j < 8; j++) {
                    const float v = (float)cd[j] * (float)sc[j];
                    x[j] = (_Float16)v;
                    y[j] = (_Float16)fmaf((float)x[j], m1, v);
                }
            } else {
                x = __builtin_bit_cast(half8, st.v[i]);
            }
            if (!plain) {
                const bool has = good >> (g >> 1) & 1;
                const int any0 = within(w.lo_any - k0) - 8 * g, any1 = within(w.hi_any - k0) - 8 * g;
                const int all0 = within(w.lo_all - k0) - 8 * g, all1 = within(w.hi_all - k0) - 8 * g;
#pragma unroll
                for (int j = 0; j < 8; j++) {
                    const bool any = has && j >= any0 && j < any1, all = has && j >= all0 && j < all1;
                    const bool inf = !__builtin_isfinite((float)x[j]);
                    odd |= inf && any && !all;
                    if (!any || (inf && !all)) {
                        x[j] = (_Float16)0.f;
                        if constexpr (Q8) y[j] = (_Float16)0.f;
                    }
                }
            }
            *reinterpret_cast<half8 *>(&T.v[0][d][8 * g]) = x;
            if constexpr (Q8) *reinterpret_cast<half8 *>(&T.v[1][d][8 * g]) = y;
        }
        if (!plain && lane == 0) T.odd[wave] = 0;
        if (odd) T.odd[wave] = 1;
        if (large) T.large = k0;
    };

    if (Q8 && tid == 0) T.large = -1;
    if (w.k0 < w.k1) load(w.k0);
    for (int k0 = w.k0; k0 < w.k1; k0 += CH) {
        const bool plain = k0 >= w.lo_all && k0 + CH <= w.hi_all && good == 15;  // uniform
        const int seen = good;
        __syncthreads();  // the last tile's reads are done
        store(k0, plain);
        __syncthreads();
        if (k0 + CH < w.k1) load(k0 + CH);
        if (!wave_on) continue;
        const int large_tile = T.large;
        // Two halves of 32 tokens: while the matrix cores have one half's scores or outputs, the
        // vector ALU has the other's softmax.  The products have priority, so that another
        // wavefront's softmax fills what they leave of the issue.
        const float mm = a.cap > 0.f ? 1.f : mul;
        const int from = within(lo - k0) - 8 * hh, end = within(hi - k0) - 8 * hh;
        // One step is two products (three: Q8_0's outputs), the read for the step after the next and
        // the part of a softmax that fits under them, in this order (the scheduler gathers the
        // products at one end otherwise).
        auto scores = [&](int u, floatx16 &s, auto under) {
            half8 kf[AHEAD + 1], qr[QL ? AHEAD + 1 : 1];
            auto read = [&](int i) { return *reinterpret_cast<const half8 *>(&T.k[32 * u + col][16 * i + 8 * hh]); };
#pragma unroll
            for (int i = 0; i < AHEAD; i++) {
                kf[i] = read(i);
                if (i < QL) qr[i] = T.ql[wave][i][lane];
            }
#pragma unroll
            for (int i = 0; i < 16; i++) s[i] = 0.f;
            floatx16 z;
            half8 sc[2];
#pragma unroll
            for (int i = 0; i < NK; i++) {
                if (i + AHEAD < NK) {
                    kf[(i + AHEAD) % (AHEAD + 1)] = read(i + AHEAD);
                    if (i + AHEAD < QL) qr[(i + AHEAD) % (AHEAD + 1)] = T.ql[wave][i + AHEAD][lane];
                }
                const half8 qlo = i < QL ? qr[i % (AHEAD + 1)] : ql[i < QL ? 0 : i - QL];
                if constexpr (Q8) {
                    if ((i & 1) == 0) {  // the first half of a block
#pragma unroll
                        for (int f = 0; f < 2; f++) sc[f] = *reinterpret_cast<const half8 *>(&T.ks[i / 2][32 * u + 16 * f + 8 * hh]);
#pragma unroll
                        for (int j = 0; j < 16; j++) z[j] = 0.f;
                    }
                    z = __builtin_amdgcn_mfma_f32_32x32x16_f16(kf[i % (AHEAD + 1)], qlo, z, 0, 0, 0);
                    z = __builtin_amdgcn_mfma_f32_32x32x16_f16(kf[i % (AHEAD + 1)], qh[i], z, 0, 0, 0);
                    under(i);
                    if (i & 1) {
#pragma unroll
                        for (int j = 0; j < 16; j++) s[j] = fmaf(z[j], (float)sc[j >> 3][j & 7], s[j]);
                    }
                } else {
                    s = __builtin_amdgcn_mfma_f32_32x32x16_f16(kf[i % (AHEAD + 1)], qlo, s, 0, 0, 0);
                    s = __builtin_amdgcn_mfma_f32_32x32x16_f16(kf[i % (AHEAD + 1)], qh[i], s, 0, 0, 0);
                    under(i);
                }
                __builtin_amdgcn_sched_barrier(0);
            }
        };
        // softcap and mask; true if the reference has to move to `mx`
        float mx;
        auto largest = [&](int u, floatx16 &s) {
            if (a.cap > 0.f) {  // uniform
#pragma unroll
                for (int i = 0; i < 16; i++) s[i] *= mul;
                cap_scores<16>(a, s);
            }
            if (!plain) {
                // register i of half hh is token 16 (i / 8) + 8 hh + i % 8 of its 32
#pragma unroll
                for (int i = 0; i < 16; i++) {
                    const int j = 32 * u + 16 * (i >> 3) + (i & 7);
                    if (!(seen >> (2 * u + (i >> 3)) & 1) || j < from || j >= end) s[i] = -INFINITY;
                }
            }
            mx = s[0];
#pragma unroll
            for (int i = 1; i < 16; i++) mx = fmaxf(mx, s[i]);
            mx = fold32(mx, MaxOp()) * mm;
            return __ballot(mx > base + 15.f) != 0;
        };
        auto rescale = [&]() {
            const float to = mx > base + 15.f ? mx - 7.f : base;  // rows that need not move stay, bit for bit
            const float alpha = base == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(base - to);
            base = to;
            l *= alpha;
#pragma unroll
            for (int d = 0; d < ND; d++)
#pragma unroll
                for (int i = 0; i < 16; i++) o[d][i] *= alpha;
        };
        // the share of step i (of NK) in the softmax of s
        auto softmax = [&](int i, floatx16 &s, half8 (&ph)[2], half8 (&pl)[2]) {
            const float sub = base == -INFINITY ? 0.f : -base;
#pragma unroll
            for (int j = 2 * (8 * i / NK); j < 2 * (8 * (i + 1) / NK); j += 2) {
                const float p0 = __builtin_amdgcn_exp2f(fmaf(s[j], mm, sub)), p1 = __builtin_amdgcn_exp2f(fmaf(s[j + 1], mm, sub));
                l += p0 + p1;
                half2_t h, r;
                split2(p0, p1, m1, h, r);
                ph[j >> 3][j & 7] = h.x, ph[j >> 3][(j & 7) + 1] = h.y;
                pl[j >> 3][j & 7] = r.x, pl[j >> 3][(j & 7) + 1] = r.y;
            }
        };
        auto outputs = [&](int u, const half8 (&ph)[2], const half8 (&pl)[2], auto under) {
            half8 vf[AHEAD + 1], vl[Q8 ? AHEAD + 1 : 1];
            auto read = [&](int plane, int i) {
                return *reinterpret_cast<const half8 *>(&T.v[plane][32 * (i % ND) + col][32 * u + 16 * (i / ND) + 8 * hh]);
            };
#pragma unroll
            for (int i = 0; i < AHEAD; i++) {
                vf[i] = read(0, i);
                if constexpr (Q8) vl[i] = read(1, i);
            }
#pragma unroll
            for (int i = 0; i < NK; i++) {
                const int f = i / ND, d = i % ND;
                if (i + AHEAD < NK) {
                    vf[(i + AHEAD) % (AHEAD + 1)] = read(0, i + AHEAD);
                    if constexpr (Q8) vl[(i + AHEAD) % (AHEAD + 1)] = read(1, i + AHEAD);
                }
                if constexpr (Q8) o[d] = __builtin_amdgcn_mfma_f32_32x32x16_f16(vl[i % (AHEAD + 1)], ph[f], o[d], 0, 0, 0);
                o[d] = __builtin_amdgcn_mfma_f32_32x32x16_f16(vf[i % (AHEAD + 1)], pl[f], o[d], 0, 0, 0);
                o[d] = __builtin_amdgcn_mfma_f32_32x32x16_f16(vf[i % (AHEAD + 1)], ph[f], o[d], 0, 0, 0);
                under(i);
                __builtin_amdgcn_sched_barrier(0);
            }
        };
        // The values under large scales, from memory: 2^-7 of one is hi + lo exactly.  Apart from the other
        // products, so that a row that does not see such a token keeps its bits.
        auto large_values = [&](int u, const half8 (&ph)[2], const half8 (&pl)[2]) {
#pragma unroll 1
            for (int f = 0; f < 2; f++) {
                const half8 pa = f ? ph[1] : ph[0], pb = f ? pl[1] : pl[0];
                const int k = k0 + 32 * u + 16 * f + 8 * hh, pk = page_of(k), slot = k & (page - 1);
                const uint8_t *p = a.kv.v + ((int64_t)(pk < 0 ? 0 : pk) * a.kv.heads + w.h) * rec;  // masked
#pragma unroll
                for (int d = 0; d < ND; d++) {
                    // addresses made here each time, not kept in registers through the main loop
                    int dim = 32 * d + col;
                    asm volatile("" : "+v"(dim));
                    const half8 cd = codes8(*reinterpret_cast<const u32x2_t *>(p + dim * page + slot));
                    const half8 sc = *reinterpret_cast<const half8 *>(p + page * D + 2 * ((dim >> 5) * page + slot));
                    half8 x, y;
#pragma unroll
                    for (int j = 0; j < 8; j++) {
                        const float v = is_large(sc[j]) ? (float)cd[j] * (float)sc[j] * 0x1p-7f : 0.f;
                        x[j] = (_Float16)v;
                        y[j] = (_Float16)fmaf((float)x[j], m1, v);
                        __builtin_amdgcn_sched_barrier(0);  // one at a time: no registers for a rare case
                    }
                    // 2^-14 of an output is exact (but for one below 2^-112)
#pragma unroll
                    for (int i = 0; i < 16; i++) o[d][i] *= 0x1p-14f;
                    o[d] = __builtin_amdgcn_mfma_f32_32x32x16_f16(y, pa, o[d], 0, 0, 0);
                    o[d] = __builtin_amdgcn_mfma_f32_32x32x16_f16(x, pb, o[d], 0, 0, 0);
                    o[d] = __builtin_amdgcn_mfma_f32_32x32x16_f16(x, pa, o[d], 0, 0, 0);
#pragma unroll
                    for (int i = 0; i < 16; i++) o[d][i] *= 0x1p14f;
                    __builtin_amdgcn_sched_barrier(0);
                }
            }
        };
        auto nothing = [](int) {};
        floatx16 s0, s1;
        half8 p0h[2], p0l[2], p1h[2], p1l[2];
        __builtin_amdgcn_s_setprio(1);
        scores(0, s0, nothing);
        __builtin_amdgcn_s_setprio(0);
        if (largest(0, s0)) rescale();
        __builtin_amdgcn_sched_barrier(0);
        __builtin_amdgcn_s_setprio(1);
        scores(1, s1, [&](int i) { softmax(i, s0, p0h, p0l); });
        // made above, not where they are used
        asm volatile("" : "+v"(p0h[0]), "+v"(p0h[1]), "+v"(p0l[0]), "+v"(p0l[1]), "+v"(l));
        __builtin_amdgcn_s_setprio(0);
        if (largest(1, s1)) {  // the first half's outputs go in under the reference they have
            outputs(0, p0h, p0l, nothing);
#pragma unroll
            for (int f = 0; f < 2; f++)
#pragma unroll
                for (int i = 0; i < 8; i++) p0h[f][i] = p0l[f][i] = (_Float16)0.f;
            rescale();
        }
        __builtin_amdgcn_sched_barrier(0);
        __builtin_amdgcn_s_setprio(1);
        outputs(0, p0h, p0l, [&](int i) { softmax(i, s1, p1h, p1l); });
        outputs(1, p1h, p1l, nothing);
        __builtin_amdgcn_s_setprio(0);
        if constexpr (Q8) {
            // rare: the probabilities once more, under the reference of the tile's end (kept until
            // here they would take 16 registers from the main loop)
            if (__builtin_amdgcn_readfirstlane(large_tile) == k0) {
                const float sum = l;
#pragma unroll 1
                for (int u = 0; u < 2; u++) {
                    scores(u, s1, nothing);
                    largest(u, s1);
#pragma unroll
                    for (int i = 0; i < NK; i++) softmax(i, s1, p1h, p1l);
                    large_values(u, p1h, p1l);
                }
                l = sum;
            }
        }
        if (!plain && (T.odd[0] | T.odd[1] | T.odd[2] | T.odd[3])) {  // rare: infinities or NaN that only some rows see
            for (int j = 0; j < CH; j++) {
                const int k = k0 + j;
                if (k >= w.lo_all && k < w.hi_all) continue;
                const int pj = page_of(k);
                if (pj < 0) continue;
                const uint8_t *p = a.kv.v + ((int64_t)pj * a.kv.heads + w.h) * rec;
                const int slot = k & (page - 1);
#pragma unroll
                for (int d = 0; d < ND; d++)
#pragma unroll
                    for (int i = 0; i < 16; i++) {
                        // addresses made here each time, not kept in registers through the main loop
                        int dim = 32 * d + 8 * (i >> 2) + 4 * hh + (i & 3);
                        asm volatile("" : "+v"(dim));
                        float y;
                        if constexpr (Q8)
                            y = (float)reinterpret_cast<const int8_t *>(p)[dim * page + slot] *
                                (float)reinterpret_cast<const _Float16 *>(p + page * D)[(dim >> 5) * page + slot];
                        else
                            y = (float)reinterpret_cast<const _Float16 *>(p)[dim * page + slot];
                        if (!__builtin_isfinite(y) && k >= lo && k < hi) o[d][i] += y;
                        __builtin_amdgcn_sched_barrier(0);  // one at a time: no registers for a rare case
                    }
            }
        }
    }
    if (!wave_on) return;
    l = fold32(l, SumOp());
    if (l != l) base = INFINITY;  // a NaN score is no maximum, but its row is not one that saw nothing
    if (!on) return;
    const int64_t rh = (int64_t)(w.nw.first + t) * a.Hq + hq;
    const bool none = base == -INFINITY;
    float f = Q8 ? 0x1p-7f : 1.f;
    float *to = a.out + rh * D;
    if (a.splits > 1) {
        const int64_t at = rh * a.splits + w.split;
        if (hh == 0) a.stat[at] = make_float2(base, l);
        if (none) return;
        to = a.part + at * D;
    } else {
        f = none ? 0.f : f / l;
    }
#pragma unroll
    for (int d = 0; d < ND; d++)
#pragma unroll
        for (int i = 0; i < 4; i++) {
            floatx4 y;
#pragma unroll
            for (int j = 0; j < 4; j++) y[j] = o[d][4 * i + j] * f;
            *reinterpret_cast<floatx4 *>(to + 32 * d + 8 * i + 4 * hh) = y;
        }
}

template <int D>
hipError_t launch_d(AttnArgs a, int dtype, int64_t blocks, hipStream_t st) {
    constexpr int64_t kBlocks = int64_t(1) << 23;
    constexpr size_t lds_q8 = sizeof(Tile<D, true>);
    constexpr size_t lds_f16 = sizeof(Tile<D, false>);
    for (int64_t b = 0; b < blocks; b += kBlocks) {
        a.block0 = b;
        const dim3 grid((unsigned)(blocks - b < kBlocks ? blocks - b : kBlocks));
        if (dtype == QMM_Q8_0) hipLaunchKernelGGL((attn_prompt_kernel<D, true>), grid, dim3(256), lds_q8, st, a);
        else hipLaunchKernelGGL((attn_prompt_kernel<D, false>), grid, dim3(256), lds_f16, st, a);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace

hipError_t launch_attn_prompt(const AttnArgs &a, int dtype, int D, int64_t blocks, hipStream_t st) {
    switch (D) {
    case 64: return launch_d<64>(a, dtype, blocks, st);
    case 96: return launch_d<96>(a, dtype, blocks, st);
    case 128: return launch_d<128>(a, dtype, blocks, st);
    case 192: return launch_d<192>(a, dtype, blocks, st);
    case 256: return launch_d<256>(a, dtype, blocks, st);
    default: return hipErrorInvalidValue;
    }
}

}  // namespace qmm
