// qmm_moe_gemm.hip -- the routed experts' products on the matrix cores, f32
// class.
//
// Exact codes, split activations.  An f32 activation row is scaled by a power
// of two so that its largest value lies in [2^9, 2^10) and split into two
// f16 numbers, x = hi + lo with |x - hi - lo| <= 2^-24 |x| (2^-25 absolute
// where lo is subnormal).  The weights enter as the integers they are made of,
// exact in f16: q - 8 (Q4_0), q (Q8_0, Q4_1), sc * q (Q4_K, Q5_K: at most
// 63 * 31 < 2^11), q - 32 (Q6_K).  v_mfma_f32_32x32x16_f16 multiplies codes by
// hi and by lo into one f32 sum per block (a chain of steps that share one
// scale), which is then scaled once in f32, as the one-token kernels do.  The
// minima of Q4_1, Q4_K and Q5_K meet the sums of x over each block (again hi +
// lo) in one more matrix step per 128 weights.  Two f16 steps per product
// against a f32 matrix step of 1/16 of their rate: f32 results at up to half
// the f16 matrix rate.
//
// Three launches: (1) qmm_moe_prep sorts the slots by expert into tiles of
// BN rows and writes the split rows; (2) moe_gemm_kernel, one workgroup per
// (row tile of the matrix, tile of slots); (3) for the down projection, the
// weighted sum over a token's slots in slot order.
#include <algorithm>

#include "qmm_device.hpp"
#include "qmm_internal.hpp"
#include "qmm_units.hpp"

namespace qmm {

namespace {

constexpr int KT = 128;                 // weights of a row per k-tile
constexpr int KT_BYTES = 4 * KT;        // a row's split activations of a k-tile: 128 hi, 128 lo
constexpr int MOE_E_MAX = QMM_MOE_MAX_EXPERTS;

// --------------------------------------------------------------- decoders ----
// The weight operand of a 32x32x16 step: lane l holds row l % 32 and, with kh
// = l / 32, 8 of the step's 16 k.  A k-tile has 8 steps; step s, half kh covers
// the 8 weights kbase(2 s + kh) + sigma(j), sigma = (0 2 1 3 4 6 5 7): the
// order in which a dword's bytes unpack pairwise.  The split activations are
// written in the same order.
//   NW          raw dwords per row and k-tile
//   STEPS       steps per chain (one scale); step(i): the i-th step to run
//   NG          load groups: group g is used up by the steps i of its eighth
//               ((i + 1) * NG / 8 > g for the first time), then reloaded with the
//               next k-tile's bytes, so a row holds one k-tile of raw registers
//   OFF         the format has block minima (offsets): one more step per tile
//   load()      group g's bytes (row offset `row` in the resource, k-tile kt)
//   scale()     the scale of the chain that step st ends; nb = blocks of 32 left in the row
//   frag()      the weight operand of step st
//   xscale(p)   factor on the activations of piece p (a power of two)
typedef _Float16 half2v __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint32_t u32(half2v v) { return __builtin_bit_cast(uint32_t, v); }
__device__ __forceinline__ half2v h2(uint32_t v) { return __builtin_bit_cast(half2v, v); }
__device__ __forceinline__ half2v splat(float v) { return half2v{(_Float16)v, (_Float16)v}; }
__device__ __forceinline__ half8 join(half2v a, half2v b, half2v c, half2v d) {
    return half8{a.x, a.y, b.x, b.y, c.x, c.y, d.x, d.y};
}
// codes of a dword's nibbles (mask 0x000F000F of w, w >> 8) as f16: 1024 + c by
// bits, then an exact subtraction
__device__ __forceinline__ half2v lo_code(uint32_t w, float bias) { return h2((w & 0x000F000Fu) | 0x64006400u) - splat(1024.f + bias); }
// high nibbles: 1024 + 16 c, so 16 (c - bias)
__device__ __forceinline__ half2v hi_code(uint32_t w, float bias) { return h2((w & 0x00F000F0u) | 0x64006400u) - splat(1024.f + 16.f * bias); }
__device__ __forceinline__ half2v byte02_code(uint32_t w, float bias) { return bytes02_as_f16(w) - splat(1024.f + bias); }
__device__ __forceinline__ half2v byte13_code(uint32_t w, float bias) { return bytes13_as_f16(w) - splat(1024.f + bias); }

__device__ __forceinline__ uint32_t ld16(Rsrc rs, uint32_t off) { return (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(rs, off, 0, 0); }
__device__ __forceinline__ u32x2_t ld64(Rsrc rs, uint32_t off) { return __builtin_amdgcn_raw_buffer_load_b64(rs, off, 0, 0); }
__device__ __forceinline__ u32x4_t ld128(Rsrc rs, uint32_t off) { return __builtin_amdgcn_raw_buffer_load_b128(rs, off, 0, 0); }

template <int DT> struct MDec;

// Q4_0, Q4_1: block b of the tile is steps 2b (low nibbles) and 2b + 1 (high
// nibbles, codes times 16, so their activations are divided by 16).
__host__ __device__ inline int kbase_nibble(int p) { return 32 * (p >> 2) + 16 * ((p >> 1) & 1) + 8 * (p & 1); }

template <> struct MDec<QMM_Q4_0> {
    static constexpr int NW = 12, STEPS = 2, NG = 4;
    static constexpr bool OFF = false;
    struct Pre {};
    __host__ __device__ static int kbase(int p) { return kbase_nibble(p); }
    __host__ __device__ static float xscale(int p) { return (p >> 1) & 1 ? 0.0625f : 1.0f; }
    __host__ __device__ static constexpr int step(int i) { return i; }
    __device__ static void load(Rsrc rs, uint32_t row, int kt, int kh, int g, uint32_t (&r)[NW]) {
        const uint32_t o = row + 72u * (uint32_t)kt + 18u * g;
        const u32x2_t q = ld64(rs, o + 2u + 8u * kh);
        r[3 * g] = q.x; r[3 * g + 1] = q.y;
        r[3 * g + 2] = ld16(rs, o);
    }
    __device__ static void prep(const uint32_t (&)[NW], int, int, Pre &) {}
    __device__ static float scale(const uint32_t (&r)[NW], int st, int nb, const Pre &) { return (st >> 1) < nb ? h2f(r[3 * (st >> 1) + 2]) : 0.f; }
    __device__ static half8 frag(const uint32_t (&r)[NW], int st, int, const Pre &) {
        const uint32_t a = r[3 * (st >> 1)], b = r[3 * (st >> 1) + 1];
        if (st & 1) return join(hi_code(a, 8.f), hi_code(a >> 8, 8.f), hi_code(b, 8.f), hi_code(b >> 8, 8.f));
        return join(lo_code(a, 8.f), lo_code(a >> 8, 8.f), lo_code(b, 8.f), lo_code(b >> 8, 8.f));
    }
};

template <> struct MDec<QMM_Q4_1> {
    static constexpr int NW = 12, STEPS = 2, NG = 4;
    static constexpr bool OFF = true;
    struct Pre { uint32_t m[4]; };
    __host__ __device__ static int kbase(int p) { return kbase_nibble(p); }
    __host__ __device__ static float xscale(int p) { return (p >> 1) & 1 ? 0.0625f : 1.0f; }
    __host__ __device__ static constexpr int step(int i) { return i; }
    __device__ static void load(Rsrc rs, uint32_t row, int kt, int kh, int g, uint32_t (&r)[NW]) {
        const uint32_t o = row + 80u * (uint32_t)kt + 20u * g;
        const u32x2_t q = ld64(rs, o + 4u + 8u * kh);
        r[3 * g] = q.x; r[3 * g + 1] = q.y;
        r[3 * g + 2] = __builtin_amdgcn_raw_buffer_load_b32(rs, o, 0, 0);
    }
    __device__ static void prep(const uint32_t (&)[NW], int, int, Pre &) {}
    // also keeps the block's minimum: the four meet [S0 S2 S1 S3] hi and lo (lane half 0)
    __device__ static float scale(const uint32_t (&r)[NW], int st, int nb, Pre &p) {
        const int b = st >> 1;
        p.m[b] = b < nb ? r[3 * b + 2] >> 16 : 0u;
        return b < nb ? h2f(r[3 * b + 2]) : 0.f;
    }
    __device__ static half8 offset(const Pre &p, float &so) {
        const half2v a = h2(p.m[0] | (p.m[2] << 16)), c = h2(p.m[1] | (p.m[3] << 16));
        so = 1.f;
        return join(a, c, a, c);
    }
    __device__ static half8 frag(const uint32_t (&r)[NW], int st, int, const Pre &) {
        const uint32_t a = r[3 * (st >> 1)], b = r[3 * (st >> 1) + 1];
        if (st & 1) return join(hi_code(a, 0.f), hi_code(a >> 8, 0.f), hi_code(b, 0.f), hi_code(b >> 8, 0.f));
        return join(lo_code(a, 0.f), lo_code(a >> 8, 0.f), lo_code(b, 0.f), lo_code(b >> 8, 0.f));
    }
};

// Q8_0: block b is steps 2b, 2b + 1; lane half kh holds bytes 16 kh .. 16 kh + 15.
template <> struct MDec<QMM_Q8_0> {
    static constexpr int NW = 20, STEPS = 2, NG = 4;
    static constexpr bool OFF = false;
    struct Pre {};
    __host__ __device__ static int kbase(int p) { return 32 * (p >> 2) + 16 * (p & 1) + 8 * ((p >> 1) & 1); }
    __host__ __device__ static float xscale(int) { return 1.0f; }
    __host__ __device__ static constexpr int step(int i) { return i; }
    __device__ static void load(Rsrc rs, uint32_t row, int kt, int kh, int g, uint32_t (&r)[NW]) {
        const uint32_t o = row + 136u * (uint32_t)kt + 34u * g;
        const u32x4_t q = ld128(rs, o + 2u + 16u * kh);
        r[5 * g] = q.x; r[5 * g + 1] = q.y; r[5 * g + 2] = q.z; r[5 * g + 3] = q.w;
        r[5 * g + 4] = ld16(rs, o);
    }
    __device__ static void prep(const uint32_t (&)[NW], int, int, Pre &) {}
    __device__ static float scale(const uint32_t (&r)[NW], int st, int nb, const Pre &) { return (st >> 1) < nb ? h2f(r[5 * (st >> 1) + 4]) : 0.f; }
    __device__ static half8 frag(const uint32_t (&r)[NW], int st, int, const Pre &) {
        const uint32_t a = r[5 * (st >> 1) + 2 * (st & 1)] ^ 0x80808080u, b = r[5 * (st >> 1) + 2 * (st & 1) + 1] ^ 0x80808080u;
        return join(byte02_code(a, 128.f), byte13_code(a, 128.f), byte02_code(b, 128.f), byte13_code(b, 128.f));
    }
};

// Q4_K, Q5_K: a k-tile is half a super-block, sub-blocks 4 (kt % 2) .. + 3: two
// chunks of 64 whose low nibbles are steps 4c, 4c + 1 and high nibbles steps
// 4c + 2, 4c + 3; lane half kh holds bytes 16 kh .. + 15 of each chunk.  The
// code enters as an f16 subnormal (c 2^-24 low, c 2^-20 high) and is multiplied
// by sc 2^10 or sc 2^6: sc * c * 2^-14, exact and never subnormal.  One chain,
// scale d 2^14.
__host__ __device__ inline int kbase_k(int p) {
    const int st = p >> 1, kh = p & 1;
    return 64 * (st >> 2) + 32 * ((st >> 1) & 1) + 16 * kh + 8 * (st & 1);
}
// four 6-bit scales (or minima) of sub-blocks 4 t .. 4 t + 3, one per byte
__device__ __forceinline__ uint32_t k_scales4(uint32_t s0, uint32_t s2, int t) {
    return t ? ((s2 & 0x0F0F0F0Fu) | ((s0 >> 2) & 0x30303030u)) : (s0 & 0x3F3F3F3Fu);
}
__device__ __forceinline__ uint32_t k_mins4(uint32_t s1, uint32_t s2, int t) {
    return t ? (((s2 >> 4) & 0x0F0F0F0Fu) | ((s1 >> 2) & 0x30303030u)) : (s1 & 0x3F3F3F3Fu);
}
template <int QH>
struct MDecK {
    static constexpr int NW = 12 + 4 * QH, STEPS = 8, NG = 2, BB = QH ? 176 : 144;
    static constexpr bool OFF = true;
    struct Pre {
        half2v a, b;  // sc of sub-blocks (0, 2) times 2^10 and (1, 3) times 2^6
        half2v m, n;  // minima of sub-blocks (0, 2) and (1, 3)
        float d, dmin;
    };
    __host__ __device__ static int kbase(int p) { return kbase_k(p); }
    __host__ __device__ static float xscale(int) { return 1.0f; }
    __host__ __device__ static constexpr int step(int i) { return i; }
    __device__ static void load(Rsrc rs, uint32_t row, int kt, int kh, int g, uint32_t (&r)[NW]) {
        const uint32_t o = row + (uint32_t)BB * (uint32_t)(kt >> 1);
        const u32x4_t q = ld128(rs, o + 16u + 32u * QH + 64u * (kt & 1) + 32u * g + 16u * kh);
        r[4 + 4 * g] = q.x; r[5 + 4 * g] = q.y; r[6 + 4 * g] = q.z; r[7 + 4 * g] = q.w;
        if (g == 0) {
            const u32x4_t h = ld128(rs, o);
            r[0] = h.x; r[1] = h.y; r[2] = h.z; r[3] = h.w;
        }
        if (QH && g == 1) {
            const u32x4_t b = ld128(rs, o + 16u + 16u * kh);
            r[NW - 4] = b.x; r[NW - 3] = b.y; r[NW - 2] = b.z; r[NW - 1] = b.w;
        }
    }
    __device__ static void prep(const uint32_t (&r)[NW], int kt, int, Pre &p) {
        const uint32_t sc = k_scales4(r[1], r[3], kt & 1), mn = k_mins4(r[2], r[3], kt & 1);
        p.a = byte02_code(sc, 0.f) * splat(1024.f);
        p.b = byte13_code(sc, 0.f) * splat(64.f);
        p.m = byte02_code(mn, 0.f);
        p.n = byte13_code(mn, 0.f);
        p.d = h2f(r[0]) * 16384.f;
        p.dmin = -h2f(r[0] >> 16);
    }
    __device__ static float scale(const uint32_t (&)[NW], int, int, const Pre &p) { return p.d; }
    __device__ static half8 offset(const Pre &p, float &so) {
        so = p.dmin;
        return join(p.m, p.n, p.m, p.n);
    }
    __device__ static half8 frag(const uint32_t (&r)[NW], int st, int kt, const Pre &p) {
        const int c = st >> 2, hi = (st >> 1) & 1, i = 4 + 4 * c + 2 * (st & 1);
        const half2v ks = hi ? p.b : p.a;
        const half2v s = c ? half2v{ks.y, ks.y} : half2v{ks.x, ks.x};
        uint32_t w[4] = {r[i], r[i] >> 8, r[i + 1], r[i + 1] >> 8};
#pragma unroll
        for (int j = 0; j < 4; j++) w[j] &= hi ? 0x00F000F0u : 0x000F000Fu;
        if constexpr (QH) {
            // bit 4 (kt % 2) + 2 c + hi of every qh byte
            const int sh = 4 * (kt & 1) + 2 * c;
            const uint32_t g0 = r[NW - 4 + 2 * (st & 1)] >> sh, g1 = r[NW - 3 + 2 * (st & 1)] >> sh;
            const uint32_t g[4] = {g0, g0 >> 8, g1, g1 >> 8};
#pragma unroll
            for (int j = 0; j < 4; j++) w[j] |= hi ? ((g[j] << 7) & 0x01000100u) : ((g[j] << 4) & 0x00100010u);
        }
        return join(h2(w[0]) * s, h2(w[1]) * s, h2(w[2]) * s, h2(w[3]) * s);
    }
};
template <> struct MDec<QMM_Q4_K> : MDecK<0> {};
template <> struct MDec<QMM_Q5_K> : MDecK<1> {};

// Q6_K: a k-tile is half h = kt % 2 of a super-block; step 2 g + li is sub-block
// 8 h + 2 g + li (16 weights l = 16 li + 8 kh + j of group g).  One chain per
// step, scale d * sc.  The steps of li = 0 run first: they use up its bytes.
template <> struct MDec<QMM_Q6_K> {
    static constexpr int NW = 15, STEPS = 1, NG = 2;
    static constexpr bool OFF = false;
    struct Pre { float s[8]; };
    __host__ __device__ static int kbase(int p) { return 8 * p; }
    __host__ __device__ static float xscale(int) { return 1.0f; }
    __host__ __device__ static constexpr int step(int i) { return 2 * (i & 3) + (i >> 2); }
    __device__ static void load(Rsrc rs, uint32_t row, int kt, int kh, int g, uint32_t (&r)[NW]) {
        const uint32_t o = row + 210u * (uint32_t)(kt >> 1), h = kt & 1;
        const u32x2_t a = ld64(rs, o + 64u * h + 16u * g + 8u * kh), b = ld64(rs, o + 64u * h + 32u + 16u * g + 8u * kh);
        const u32x2_t c = ld64(rs, o + 128u + 32u * h + 16u * g + 8u * kh);
        r[6 * g] = a.x; r[6 * g + 1] = a.y; r[6 * g + 2] = b.x; r[6 * g + 3] = b.y; r[6 * g + 4] = c.x; r[6 * g + 5] = c.y;
        if (g == 0) {
            const u32x2_t sc = ld64(rs, o + 192u + 8u * h);
            r[12] = sc.x; r[13] = sc.y;
            r[14] = ld16(rs, o + 208u);
        }
    }
    __device__ static void prep(const uint32_t (&r)[NW], int, int, Pre &p) {
        const float d = h2f(r[14]);
#pragma unroll
        for (int i = 0; i < 8; i++) p.s[i] = d * (float)(int)(int8_t)(uint8_t)(r[12 + (i >> 2)] >> (8 * (i & 3)));
    }
    __device__ static float scale(const uint32_t (&)[NW], int st, int, const Pre &p) { return p.s[st]; }
    __device__ static half8 frag(const uint32_t (&r)[NW], int st, int, const Pre &) {
        const int g = st >> 1, li = st & 1;
        uint32_t q[2];
#pragma unroll
        for (int j = 0; j < 2; j++) {
            const uint32_t l = r[6 * li + 2 * (g & 1) + j], c = r[6 * li + 4 + j];
            const uint32_t hi = (g < 2 ? (c << (4 - 2 * g)) : (c >> (2 * g - 4))) & 0x30303030u;
            q[j] = ((g < 2 ? l : l >> 4) & 0x0F0F0F0Fu) | hi;
        }
        return join(byte02_code(q[0], 32.f), byte13_code(q[0], 32.f), byte02_code(q[1], 32.f), byte13_code(q[1], 32.f));
    }
};

// ------------------------------------------------------------- preparation ----
// The workspace of one call (see moe_ws).  tiles[0].x = number of tiles; tile i
// is tiles[1 + i] = (expert, first position in order, rows, 0).
struct MoeWs {
    int4 *tiles;
    int32_t *order;   // the slots, expert after expert
    float *rscale;    // per row: what the split row was divided by
    uint4 *sums;      // [row][k-tile]: 4 block sums, hi and lo (formats with minima)
    uint8_t *xs;      // [row][k-tile][KT_BYTES]
    float *prod;      // down: [slot][M]
};

// Block 0 sorts the S slots by expert and cuts each expert's run into tiles of
// BN; the order of slots within an expert moves no result (every output row
// depends on its own activation row alone).
__device__ void plan_tiles(const int32_t *ids, int S, int E, int BN, int4 *tiles, int32_t *order) {
    __shared__ int count[MOE_E_MAX], start[MOE_E_MAX + 1], tile0[MOE_E_MAX + 1];
    const int t = (int)threadIdx.x, T = (int)blockDim.x;
    for (int e = t; e < E; e += T) count[e] = 0;
    __syncthreads();
    for (int s = t; s < S; s += T) {
        const int e = ids[s];
        if (e >= 0 && e < E) atomicAdd(&count[e], 1);
    }
    __syncthreads();
    if (t < 64) {  // one wavefront: exclusive sums over the experts, 64 at a time
        int base = 0, tbase = 0;
        for (int e0 = 0; e0 < E; e0 += 64) {
            const int c = e0 + t < E ? count[e0 + t] : 0, tc = (c + BN - 1) / BN;
            int v = c, w = tc;
#pragma unroll
            for (int o = 1; o < 64; o <<= 1) {
                const int a = __shfl_up(v, o, 64), b = __shfl_up(w, o, 64);
                if (t >= o) { v += a; w += b; }
            }
            if (e0 + t < E) {
                start[e0 + t] = base + v - c;
                tile0[e0 + t] = tbase + w - tc;
            }
            base += __shfl(v, 63, 64);
            tbase += __shfl(w, 63, 64);
        }
        if (t == 0) tiles[0] = int4{tbase, 0, 0, 0};
    }
    __syncthreads();
    for (int e = t; e < E; e += T) {
        const int c = count[e];
        for (int i = 0; i * BN < c; i++)
            tiles[1 + tile0[e] + i] = int4{e, start[e] + i * BN, c - i * BN < BN ? c - i * BN : BN, 0};
    }
    __syncthreads();
    for (int s = t; s < S; s += T) {
        const int e = ids[s];
        if (e >= 0 && e < E) order[atomicAdd(&start[e], 1)] = s;
    }
}

// Blocks 1 ..: one activation row each (rows of a slot without an expert are
// skipped where skip_ids is given).  Threads hold 8 values per piece.
template <int DT>
__global__ void __launch_bounds__(256) moe_prep_kernel(const int32_t *ids, int S, int E, int BN, MoeWs ws, const float *X,
                                                       int64_t rows, int K, int nkt, int per_row_ids) {
    if (blockIdx.x == 0) {
        plan_tiles(ids, S, E, BN, ws.tiles, ws.order);
        return;
    }
    const int64_t row = (int64_t)blockIdx.x - 1;
    if (per_row_ids) {
        const int e = ids[row];
        if (e < 0 || e >= E) return;
    }
    const float *x = X + row * K;
    const int t = (int)threadIdx.x, T = (int)blockDim.x;
    __shared__ float red[4];
    float amax = 0.f;
    for (int i = t; i < K / 4; i += T) {  // K % 32 == 0
        const floatx4 v = reinterpret_cast<const floatx4 *>(x)[i];
#pragma unroll
        for (int j = 0; j < 4; j++) {
            const float a = fabsf(v[j]);
            amax = (a > amax && a < __builtin_inff()) ? a : amax;
        }
    }
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor(amax, o, 64));
    if ((t & 63) == 0) red[t >> 6] = amax;
    __syncthreads();
    amax = red[0];
    for (int w = 1; w < T / 64; w++) amax = fmaxf(amax, red[w]);
    // amax = f * 2^e, f in [0.5, 1): multiply by 2^(10 - e)
    int e = 0;
    (void)frexpf(amax, &e);
    int m = amax > 0.f ? 10 - e : 0;
    m = m > 126 ? 126 : m;
    const float mul = ldexpf(1.0f, m);
    if (t == 0) ws.rscale[row] = ldexpf(1.0f, -m);
    uint8_t *dst = ws.xs + row * (int64_t)nkt * KT_BYTES;
    for (int i = t; i < nkt * 16; i += T) {
        const int kt = i >> 4, p = i & 15, k = kt * KT + MDec<DT>::kbase(p);
        const float f = mul * MDec<DT>::xscale(p);
        float v[8];
        float sum = 0.f;
        if (k < K) {  // whole pieces: K % 32 == 0
            const floatx4 a = *reinterpret_cast<const floatx4 *>(x + k), b = *reinterpret_cast<const floatx4 *>(x + k + 4);
            v[0] = a.x; v[1] = a.z; v[2] = a.y; v[3] = a.w; v[4] = b.x; v[5] = b.z; v[6] = b.y; v[7] = b.w;
#pragma unroll
            for (int j = 0; j < 8; j++) sum += mul * v[j];
        } else {
#pragma unroll
            for (int j = 0; j < 8; j++) v[j] = 0.f;
        }
        half8 hi, lo;
#pragma unroll
        for (int j = 0; j < 8; j++) {
            const float s = v[j] * f;
            hi[j] = (_Float16)s;
            const float r = s - (float)hi[j];
            lo[j] = (_Float16)(r == r ? r : 0.f);  // a non-finite x is in hi alone
        }
        reinterpret_cast<half8 *>(dst + (int64_t)kt * KT_BYTES)[p] = hi;
        reinterpret_cast<half8 *>(dst + (int64_t)kt * KT_BYTES)[16 + p] = lo;
        if constexpr (MDec<DT>::OFF) {
            // block b's four pieces: 4b .. 4b+3 (Q4_1) or, for the K formats,
            // 8 (b >> 1) + 4 (b & 1) .. + 3: four neighbouring lanes either way
            sum += __shfl_xor(sum, 1, 64);
            sum += __shfl_xor(sum, 2, 64);
            const float s0 = __shfl(sum, (t & 48) + 0, 64), s1 = __shfl(sum, (t & 48) + 4, 64);
            const float s2 = __shfl(sum, (t & 48) + 8, 64), s3 = __shfl(sum, (t & 48) + 12, 64);
            if (p == 0) {
                const float s[4] = {s0, s2, s1, s3};
                half8 o;
#pragma unroll
                for (int j = 0; j < 4; j++) {
                    o[j] = (_Float16)s[j];
                    const float r = s[j] - (float)o[j];
                    o[4 + j] = (_Float16)(r == r ? r : 0.f);
                }
                ws.sums[row * nkt + kt] = __builtin_bit_cast(uint4, o);
            }
        }
    }
}

// ------------------------------------------------------------------- GEMM ----
struct MoeGemmArgs {
    const uint8_t *w0, *w1;  // swiglu: gate and up; down: w0 alone
    MoeWs ws;
    float *out;              // swiglu: out[slot][M]; down: prod[slot][M]
    int64_t M, row_bytes, mat_bytes;
    int K, nkt, mtiles, T;   // T: slots per activation row (1 when every slot has its own)
    uint32_t xs_bytes;       // of ws.xs
};

// A workgroup: W wavefronts, each 2 x 32 rows (swiglu: 32 gate rows and the
// same 32 up rows) against the BN = 32 FN slots of a tile.
template <int DT, int FN, int W, bool SWI>
__global__ void __launch_bounds__(64 * W, 2) moe_gemm_kernel(const MoeGemmArgs a) {
    using D = MDec<DT>;
    constexpr int BN = 32 * FN, RW = SWI ? 32 : 64, BM = RW * W;
    constexpr int NP = BN * 32 / (64 * W);  // 16-byte pieces of a k-tile per thread
    static_assert(NP >= 1, "tile too small for the workgroup");
    __shared__ __attribute__((aligned(16))) uint8_t xl[2][BN * KT_BYTES];
    __shared__ int32_t slot_of[BN];
    __shared__ float rsc[BN];
    const int t = (int)threadIdx.x, lane = t & 63, wave = __builtin_amdgcn_readfirstlane(t >> 6);
    const int l32 = lane & 31, kh = lane >> 5;

    // workgroups of one XCD (id mod 8) take neighbouring tiles of slots for
    // the same rows of the matrix: the slots of an expert meet in one L2
    const int nt = a.ws.tiles[0].x, total = nt * a.mtiles, chunk = (total + 7) / 8;
    const int id = ((int)blockIdx.x & 7) * chunk + ((int)blockIdx.x >> 3);
    if (((int)blockIdx.x >> 3) >= chunk || id >= total) return;
    const int mt = id / nt;
    const int4 tile = a.ws.tiles[1 + id % nt];
    const int e = __builtin_amdgcn_readfirstlane(tile.x), n_rows = __builtin_amdgcn_readfirstlane(tile.z);
    for (int i = t; i < BN; i += 64 * W) {
        const int s = i < n_rows ? a.ws.order[tile.y + i] : -1;
        slot_of[i] = s;
        rsc[i] = s >= 0 ? a.ws.rscale[s / a.T] : 0.f;
    }
    __syncthreads();

    // activation pieces: piece c of thread t is 16-byte piece t % 32 of row t / 32 + c (2 W)
    uint32_t xoff[NP];
    uint32_t xdst[NP];
#pragma unroll
    for (int c = 0; c < NP; c++) {
        const int r = (t >> 5) + c * (2 * W), p = t & 31;
        const int s = slot_of[r];
        // rows past the tile's end read nothing (zeros)
        xoff[c] = s >= 0 ? (uint32_t)(s / a.T) * (uint32_t)(a.nkt * KT_BYTES) + 16u * p : 0xFFFFFFF0u - (uint32_t)(a.nkt * KT_BYTES);
        xdst[c] = (uint32_t)(r * KT_BYTES + 16 * ((p & 16) | ((p ^ r) & 15)));
    }
    const Rsrc xrs = make_rsrc_uniform(a.ws.xs, a.xs_bytes);

    // this wavefront's rows of the matrix
    const int64_t m0 = (int64_t)mt * BM + (SWI ? 32 * wave : 64 * wave);
    const int64_t left = a.M - m0;  // rows that exist (may be <= 0)
    const int64_t base = (int64_t)e * a.mat_bytes + (left > 0 ? m0 : 0) * a.row_bytes;
    const uint32_t mis = (uint32_t)(base & 3);  // the resource starts on a dword
    const uint32_t nb0 = left > 0 ? (uint32_t)((left < RW ? left : RW) * a.row_bytes) + mis : 0u;
    const Rsrc wr0 = make_rsrc_uniform(a.w0 + (base - mis), nb0);
    const Rsrc wr1 = SWI ? make_rsrc_uniform(a.w1 + (base - mis), nb0) : wr0;
    const uint32_t ro0 = mis + (uint32_t)l32 * (uint32_t)a.row_bytes;
    const uint32_t ro1 = SWI ? ro0 : ro0 + 32u * (uint32_t)a.row_bytes;

    // block sums of the lane's slots (formats with minima): lane half 0 alone
    const uint4 *sump[FN];
    if constexpr (D::OFF) {
#pragma unroll
        for (int f = 0; f < FN; f++) {
            const int s = slot_of[32 * f + l32];
            sump[f] = a.ws.sums + (int64_t)(s >= 0 ? s / a.T : 0) * a.nkt;
        }
    }

    floatx16 acc[2][FN];
#pragma unroll
    for (int i = 0; i < 2; i++)
#pragma unroll
        for (int f = 0; f < FN; f++)
#pragma unroll
            for (int j = 0; j < 16; j++) acc[i][f][j] = 0.f;

    uint32_t raw[2][D::NW];
    u32x4_t xr[(NP + 1) / 2];
    auto fetch_w = [&](int kt, int g) {
        D::load(wr0, ro0, kt, kh, g, raw[0]);
        D::load(wr1, ro1, kt, kh, g, raw[1]);
    };
    // the activations of a k-tile move in two halves through registers
    auto fetch_x = [&](int kt, int h) {
#pragma unroll
        for (int c = 0; c < NP; c++)
            if (c * 2 / NP == h) xr[c % ((NP + 1) / 2)] = __builtin_amdgcn_raw_buffer_load_b128(xrs, xoff[c], (uint32_t)(kt * KT_BYTES), 0);
    };
    auto store_x = [&](int buf, int h) {
#pragma unroll
        for (int c = 0; c < NP; c++)
            if (c * 2 / NP == h) *reinterpret_cast<u32x4_t *>(&xl[buf][xdst[c]]) = xr[c % ((NP + 1) / 2)];
    };
#pragma unroll
    for (int h = 0; h < 2; h++) {
        fetch_x(0, h);
        store_x(0, h);
    }
#pragma unroll
    for (int g = 0; g < D::NG; g++) fetch_w(0, g);
    __syncthreads();

    for (int kt = 0; kt < a.nkt; kt++) {
        const int buf = kt & 1;
        // the next k-tile's loads (past the last one: the last again, unused)
        const int kn = kt + 1 < a.nkt ? kt + 1 : kt;
        fetch_x(kn, 0);
        half8 so_a[FN];
        if constexpr (D::OFF) {
#pragma unroll
            for (int f = 0; f < FN; f++) {
                const uint4 v = sump[f][kt];
                so_a[f] = kh == 0 ? __builtin_bit_cast(half8, v) : half8{0, 0, 0, 0, 0, 0, 0, 0};
            }
        }
        const int nb = (a.K - kt * KT) / 32;
        typename D::Pre pre[2];
#pragma unroll
        for (int i = 0; i < 2; i++) D::prep(raw[i], kt, nb, pre[i]);
        const uint8_t *xb = &xl[buf][l32 * KT_BYTES];
        floatx16 tmp[2][FN];
#pragma unroll
        for (int n = 0; n < 8; n++) {
            const int st = D::step(n);
            half8 b[2];
#pragma unroll
            for (int i = 0; i < 2; i++) b[i] = D::frag(raw[i], st, kt, pre[i]);
            const int p = ((2 * st + kh) ^ l32) & 15;
#pragma unroll
            for (int f = 0; f < FN; f++) {
                const half8 ah = *reinterpret_cast<const half8 *>(xb + 32 * f * KT_BYTES + 16 * p);
                const half8 al = *reinterpret_cast<const half8 *>(xb + 32 * f * KT_BYTES + 256 + 16 * p);
#pragma unroll
                for (int i = 0; i < 2; i++) {
                    if (n % D::STEPS == 0) {
                        floatx16 z;
#pragma unroll
                        for (int j = 0; j < 16; j++) z[j] = 0.f;
                        tmp[i][f] = __builtin_amdgcn_mfma_f32_32x32x16_f16(al, b[i], z, 0, 0, 0);
                    } else {
                        tmp[i][f] = __builtin_amdgcn_mfma_f32_32x32x16_f16(al, b[i], tmp[i][f], 0, 0, 0);
                    }
                    tmp[i][f] = __builtin_amdgcn_mfma_f32_32x32x16_f16(ah, b[i], tmp[i][f], 0, 0, 0);
                }
            }
            if ((n + 1) % D::STEPS == 0) {
                // the end of a chain: scale its sum once, in f32
#pragma unroll
                for (int i = 0; i < 2; i++) {
                    const float s = D::scale(raw[i], st, nb, pre[i]);
#pragma unroll
                    for (int f = 0; f < FN; f++)
#pragma unroll
                        for (int j = 0; j < 16; j++) acc[i][f][j] = fmaf(s, tmp[i][f][j], acc[i][f][j]);
                }
            }
            if ((n + 1) % (8 / D::NG) == 0) fetch_w(kn, n / (8 / D::NG));
            if (n == 3) {
                store_x(buf ^ 1, 0);
                fetch_x(kn, 1);
            }
            // one chain's sums at a time: left alone the compiler starts
            // several and spills them
            if ((n + 1) % D::STEPS == 0 || n == 3) __builtin_amdgcn_sched_barrier(0);
        }
        if constexpr (D::OFF) {
#pragma unroll
            for (int i = 0; i < 2; i++) {
                float so;
                const half8 off = D::offset(pre[i], so);
#pragma unroll
                for (int f = 0; f < FN; f++) {
                    floatx16 z;
#pragma unroll
                    for (int j = 0; j < 16; j++) z[j] = 0.f;
                    z = __builtin_amdgcn_mfma_f32_32x32x16_f16(so_a[f], off, z, 0, 0, 0);
#pragma unroll
                    for (int j = 0; j < 16; j++) acc[i][f][j] = fmaf(so, z[j], acc[i][f][j]);
                }
            }
        }
        store_x(buf ^ 1, 1);
        __syncthreads();
    }

    // lane: matrix row m0 + l32 (+ 32); register j: slot 8 (j / 4) + 4 kh + j % 4 of the tile
#pragma unroll
    for (int f = 0; f < FN; f++)
#pragma unroll
        for (int j = 0; j < 16; j++) {
            const int r = 32 * f + 8 * (j >> 2) + 4 * kh + (j & 3);
            const int64_t s = slot_of[r];
            const float sc = rsc[r];
            if (s >= 0) {
                if constexpr (SWI) {
                    if (l32 < left) a.out[s * a.M + m0 + l32] = silu(acc[0][f][j] * sc) * (acc[1][f][j] * sc);
                } else {
                    if (l32 < left) a.out[s * a.M + m0 + l32] = acc[0][f][j] * sc;
                    if (l32 + 32 < left) a.out[s * a.M + m0 + 32 + l32] = acc[1][f][j] * sc;
                }
            }
        }
}

// out[slot][:] = 0 where a slot has no expert (the GEMM writes no such row)
__global__ void __launch_bounds__(256) moe_zero_kernel(const int32_t *ids, int E, int64_t M, float *out) {
    const int64_t s = blockIdx.x;
    const int e = ids[s];
    if (e >= 0 && e < E) return;
    for (int64_t m = threadIdx.x; m < M; m += 256) out[s * M + m] = 0.f;
}

// Y[n][m] = residual[n][m] + sum over t of weights[n][t] * prod[n T + t][m]
__global__ void __launch_bounds__(256) moe_combine_kernel(const int32_t *ids, const float *weights, const float *prod,
                                                          const float *residual, float *Y, int E, int64_t M, int T) {
    const int64_t n = blockIdx.x;
    for (int64_t m = (int64_t)blockIdx.y * 256 + threadIdx.x; m < M; m += (int64_t)gridDim.y * 256) {
        float y = residual ? residual[n * M + m] : 0.f;
        for (int t = 0; t < T; t++) {
            const int e = ids[n * T + t];
            if (e >= 0 && e < E) y = fmaf(weights[n * T + t], prod[(n * T + t) * M + m], y);
        }
        Y[n * M + m] = y;
    }
}

// --------------------------------------------------------------- launchers ----
constexpr int64_t align256(int64_t v) { return (v + 255) & ~(int64_t)255; }

// Tokens per pass: the split rows stay below 2^31 bytes (32-bit offsets), the
// down products below 1 GB; longer inputs run pass after pass in one workspace.
int64_t chunk_tokens(int64_t K, int64_t M, int64_t N, int64_t T, bool down) {
    const int64_t nkt = (K + KT - 1) / KT, row = nkt * KT_BYTES;
    int64_t n = (int64_t(1) << 30) / (down ? row * T : row);
    if (down) n = std::min(n, (int64_t(1) << 30) / (4 * M * T));
    n = std::min(n, (int64_t(1) << 22) / T);  // slots: grids of 2^32 threads
    n = std::min(n, (int64_t(1) << 27) / T / (M / 64 + 1));  // (tiles of 32 slots) x (tiles of 128 rows) <= 2^23
    return std::max<int64_t>(1, std::min(n, N));
}

struct MoeSizes {
    int64_t tokens, slots, rows, nkt, tiles;
    int64_t o_order, o_rscale, o_sums, o_xs, o_prod, bytes;
};
MoeSizes moe_sizes(int dtype, int64_t E, int64_t M, int64_t K, int64_t N, int64_t T, int BN, bool down) {
    MoeSizes z;
    z.tokens = chunk_tokens(K, M, N, T, down);
    z.slots = z.tokens * T;
    z.rows = down ? z.slots : z.tokens;
    z.nkt = (K + KT - 1) / KT;
    z.tiles = z.slots / BN + std::min(E, z.slots);
    const bool off = dtype == QMM_Q4_1 || dtype == QMM_Q4_K || dtype == QMM_Q5_K;
    z.o_order = align256(16 * (1 + z.tiles));
    z.o_rscale = z.o_order + align256(4 * z.slots);
    z.o_sums = z.o_rscale + align256(4 * z.rows);
    z.o_xs = z.o_sums + (off ? align256(16 * z.rows * z.nkt) : 0);
    z.o_prod = z.o_xs + align256(z.rows * z.nkt * KT_BYTES);
    z.bytes = z.o_prod + (down ? align256(4 * z.slots * M) : 0);
    return z;
}

template <int DT, int FN, int W, bool SWI>
void launch_gemm(const MoeGemmArgs &a, int64_t tiles, hipStream_t st) {
    const int64_t blocks = (tiles * a.mtiles + 7) / 8 * 8;
    hipLaunchKernelGGL((moe_gemm_kernel<DT, FN, W, SWI>), dim3((unsigned)blocks), dim3(64 * W), 0, st, a);
}

template <int DT, bool SWI>
hipError_t run_gemm(const void *w0, const void *w1, int64_t E, int64_t M, int64_t K, int64_t N, int64_t T, const int32_t *ids,
                    const float *weights, const float *X, const float *residual, float *out, void *work, hipStream_t st) {
    constexpr int W = 4;
    const int BN = moe_gemm_bn(E, N, T);
    const MoeSizes z = moe_sizes(DT, E, M, K, N, T, BN, !SWI);
    uint8_t *p = static_cast<uint8_t *>(work);
    MoeGemmArgs a;
    a.w0 = static_cast<const uint8_t *>(w0);
    a.w1 = static_cast<const uint8_t *>(w1);
    a.ws = {reinterpret_cast<int4 *>(p), reinterpret_cast<int32_t *>(p + z.o_order), reinterpret_cast<float *>(p + z.o_rscale),
            reinterpret_cast<uint4 *>(p + z.o_sums), p + z.o_xs, reinterpret_cast<float *>(p + z.o_prod)};
    a.M = M;
    a.row_bytes = K / Geo<DT>::BS * Geo<DT>::BB;
    a.mat_bytes = M * a.row_bytes;
    a.K = (int)K;
    a.nkt = (int)z.nkt;
    a.mtiles = (int)((M + (SWI ? 32 : 64) * W - 1) / ((SWI ? 32 : 64) * W));
    a.T = SWI ? (int)T : 1;
    for (int64_t n0 = 0; n0 < N; n0 += z.tokens) {
        const int64_t n = std::min(z.tokens, N - n0), S = n * T, rows = SWI ? n : S;
        const int32_t *idc = ids + n0 * T;
        a.xs_bytes = (uint32_t)(rows * z.nkt * KT_BYTES);
        a.out = SWI ? out + n0 * T * M : a.ws.prod;
        hipLaunchKernelGGL((moe_prep_kernel<DT>), dim3((unsigned)(rows + 1)), dim3(256), 0, st, idc, (int)S, (int)E, BN, a.ws, X + n0 * (SWI ? 1 : T) * K, rows, (int)K, (int)z.nkt, SWI ? 0 : 1);
        const int64_t tiles = S / BN + std::min(E, S);
        if (BN == 32) launch_gemm<DT, 1, W, SWI>(a, tiles, st);
        else launch_gemm<DT, 2, W, SWI>(a, tiles, st);
        if (SWI) {
            hipLaunchKernelGGL(moe_zero_kernel, dim3((unsigned)S), dim3(256), 0, st, idc, (int)E, M, a.out);
        } else {
            const unsigned gy = (unsigned)std::min<int64_t>((M + 255) / 256, 64);
            hipLaunchKernelGGL(moe_combine_kernel, dim3((unsigned)n, gy), dim3(256), 0, st, idc, weights + n0 * T, a.ws.prod,
                               residual ? residual + n0 * M : nullptr, out + n0 * M, (int)E, M, (int)T);
        }
    }
    return hipGetLastError();
}

}  // namespace

// Slots per tile: 32 while an expert sees few of them, else 64.
int moe_gemm_bn(int64_t E, int64_t N, int64_t T) { return N * T <= 32 * E ? 32 : 64; }

int64_t moe_gemm_work_bytes(int dtype, int64_t E, int64_t M, int64_t K, int64_t N, int64_t T, bool down) {
    return moe_sizes(dtype, E, M, K, N, T, moe_gemm_bn(E, N, T), down).bytes;
}

hipError_t launch_moe_gemm_swiglu(const void *gate, const void *up, int dtype, int64_t E, int64_t M, int64_t K, int64_t N,
                                  int64_t T, const int32_t *ids, const float *X, float *out, void *work, hipStream_t st) {
#define QMM_CALL(DT) return run_gemm<DT, true>(gate, up, E, M, K, N, T, ids, nullptr, X, nullptr, out, work, st)
    QMM_MOE_DT(dtype, QMM_CALL)
#undef QMM_CALL
    return hipErrorInvalidValue;
}

hipError_t launch_moe_gemm_down(const void *w, int dtype, int64_t E, int64_t M, int64_t K, int64_t N, int64_t T,
                                const int32_t *ids, const float *weights, const float *H, const float *residual, float *Y,
                                void *work, hipStream_t st) {
#define QMM_CALL(DT) return run_gemm<DT, false>(w, nullptr, E, M, K, N, T, ids, weights, H, residual, Y, work, st)
    QMM_MOE_DT(dtype, QMM_CALL)
#undef QMM_CALL
    return hipErrorInvalidValue;
}

}  // namespace qmm
