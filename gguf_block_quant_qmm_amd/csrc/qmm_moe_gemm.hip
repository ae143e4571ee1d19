// qmm_moe_gemm.hip -- the routed experts' products on the matrix cores, f32
// class.
//
// Exact codes, split activations.  An f32 activation row is scaled by a power
// of two so that its largest value lies in [2^9, 2^10) and split into two
// f16 numbers, x = hi + lo with |x - hi - lo| <= 2^-23 |x| (what an 11-bit hi
// leaves of 24 bits takes up to 12, lo holds 11), or 2^-25 absolute where lo is
// subnormal; high nibbles of Q4_0 and Q4_1 enter as 16 times their code against
// x / 16, where that is 2^-21, at most 2^-30 of the row's largest value.  The
// weights enter as the integers they are made of,
// exact in f16: q - 8 (Q4_0), q (Q8_0, Q4_1), sc * q (Q4_K, Q5_K: at most
// 63 * 31 < 2^11), q - 32 (Q6_K).  v_mfma_f32_32x32x16_f16 multiplies codes by
// hi and by lo into one f32 sum per block (a chain of steps that share one
// scale), which is then scaled once in f32, as the one-token kernels do.  The
// minima of Q4_1, Q4_K and Q5_K meet the sums of x over each block (again hi +
// lo) in one more matrix step per 128 weights.  Two f16 steps per product
// against a f32 matrix step of 1/16 of their rate: f32 results at up to half
// the f16 matrix rate.
//
// Three launches: (1) moe_prep_kernel sorts the slots by expert into tiles of
// BN rows and writes the split rows; (2) moe_gemm_kernel, one workgroup per
// (row tile of the matrix, tile of slots, share of K); (3) for the down
// projection, the weighted sum over a token's slots in slot order (for gate/up
// with a shared K, silu(gate) * up of the summed shares).
//
// Measured (profiler's medians of launch (2), the experts' tensors rotating through
// 1 GiB), 512 tokens, gate/up of 2 of 8 experts 14336 x 4096: Q4_K 593-626 us (the
// clock drops for the first dozens of launches), 384-405 TFLOP/s of the formula's
// operations, twice that of the matrix cores' (a large f16 product reaches 1130-1280
// here); Q4_0 619, Q4_1 652, Q5_K 661, Q8_0 734, Q6_K 846.  512 tokens, 8 of 64
// experts, Q8_0: gate/up 1024 x 4096 301-339 us, down 4096 x 1024 144-163.  37
// tokens, gate/up of 4 of 60 experts 1408 x 2048 Q6_K, 83.  It is a sum, not an
// overlap: the Q4_K case keeps the matrix cores busy for 235 us and issues VALU
// instructions for 183, along two barriers per k-tile.  Taken out one at a time, it
// lost, at 640 us, 113 us with the weights' loads and stores, 75 with the
// activations', 47 with the barriers, 47 with the minima, 13 with the decoding; the
// matrix steps and the barriers alone take 412.  Launch (1) takes 6 us there, and 80
// for 4096 tokens of 8 slots, where one workgroup's plan outlasts the row split.
// Times of two variants beside each other below are from a captured graph over four
// inputs.
#include <algorithm>

#include "qmm_device.hpp"
#include "qmm_internal.hpp"
#include "qmm_units.hpp"

namespace qmm {

namespace {

constexpr int KT = 128;                 // weights of a row per k-tile
constexpr int XT_BYTES = 2 * KT;        // a row's split activations of half a k-tile: 64 hi, 64 lo
constexpr int KT_BYTES = 2 * XT_BYTES;
constexpr int WL_ROWS = 74;             // rows of a wavefront in LDS: 64, and those a half's last load has too many
constexpr int MOE_E_MAX = QMM_MOE_MAX_EXPERTS;

// --------------------------------------------------------------- decoders ----
// The weight operand of a 32x32x16 step: lane l holds row l % 32 and, with kh
// = l / 32, 8 of the step's 16 k.  A k-tile has 8 steps; step s, half kh covers
// the 8 weights kbase(2 s + kh) + sigma(j), sigma = (0 2 1 3 4 6 5 7): the
// order in which a dword's bytes unpack pairwise.  The split activations are
// written in the same order.
//   LP          pieces of 16 bytes that a row's k-tile is loaded in, one lane each:
//               everything a step needs, headers and scales too: loaded by instructions
//               of their own these touch every cache line again (gate/up of 8 tokens, 2
//               of 8 experts 14336 x 4096: Q6_K 260 us against 291, Q8_0 254 / 279,
//               Q5_K 213 / 240, Q4_K 180 / 186)
//   TB, at, odd piece j of k-tile kt of a row: byte TB(kt) + at(j), + odd(j) for odd kt
//   ROW         bytes a row's pieces take in LDS, back to back (a multiple of 16 whose
//               dwords step through all banks: 16 rows' 16-byte reads never collide)
//   NW          raw dwords per row and k-tile in registers
//   STEPS       steps per chain (one scale); step(i): the i-th step to run
//   NG          groups of raw dwords, group g read from LDS while group g - 1 runs
//   OFF         the format has block minima (offsets): one more step per tile
//   EARLY       nothing is read from LDS after the last step's operand
//   read()      group g of a row from LDS
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

__device__ __forceinline__ uint32_t ld16(Rsrc rs, uint32_t off, uint32_t so) { return (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(rs, off, so, 0); }
__device__ __forceinline__ uint32_t ld32(Rsrc rs, uint32_t off, uint32_t so) { return __builtin_amdgcn_raw_buffer_load_b32(rs, off, so, 0); }
__device__ __forceinline__ u32x4_t ld128(Rsrc rs, uint32_t off, uint32_t so) { return __builtin_amdgcn_raw_buffer_load_b128(rs, off, so, 0); }
__device__ __forceinline__ uint32_t at32(const uint8_t *p) { return *reinterpret_cast<const uint32_t *>(p); }
__device__ __forceinline__ uint32_t at16(const uint8_t *p) { return *reinterpret_cast<const uint16_t *>(p); }
__device__ __forceinline__ u32x2_t at64(const uint8_t *p) { return *reinterpret_cast<const u32x2_t *>(p); }
__device__ __forceinline__ u32x4_t at128(const uint8_t *p) { return *reinterpret_cast<const u32x4_t *>(p); }
// 4 N bytes at p, a dword boundary or 2 past one
template <int N, bool ODD>
__device__ __forceinline__ void lds_dwords(const uint8_t *p, uint32_t *r) {
    uint32_t w[N + 1];
#pragma unroll
    for (int i = 0; i < N + (ODD ? 1 : 0); i++) w[i] = at32(p - (ODD ? 2 : 0) + 4 * i);
#pragma unroll
    for (int i = 0; i < N; i++) r[i] = ODD ? __builtin_amdgcn_alignbyte(w[i + 1], w[i], 2) : w[i];
}

template <int DT> struct MDec;

// Q4_0, Q4_1: block b of the tile is steps 2b (low nibbles) and 2b + 1 (high
// nibbles, codes times 16, so their activations are divided by 16).
__host__ __device__ inline int kbase_nibble(int p) { return 32 * (p >> 2) + 16 * ((p >> 1) & 1) + 8 * (p & 1); }

template <> struct MDec<QMM_Q4_0> {
    static constexpr int NW = 12, STEPS = 2, NG = 4;
    static constexpr bool OFF = false, EARLY = true;
    struct Pre {};
    __host__ __device__ static int kbase(int p) { return kbase_nibble(p); }
    __host__ __device__ static float xscale(int p) { return (p >> 1) & 1 ? 0.0625f : 1.0f; }
    __host__ __device__ static constexpr int step(int i) { return i; }
    static constexpr int LP = 5, ROW = 80;  // 72 bytes
    __device__ static uint32_t TB(int kt) { return 72u * (uint32_t)kt; }
    __device__ static uint32_t at(int j) { return 16u * (uint32_t)j; }
    __device__ static uint32_t odd(int) { return 0u; }
    __device__ static void read(const uint8_t *p, int kh, int g, uint32_t (&r)[NW]) {
        if (g & 1) lds_dwords<2, false>(p + 18 * g + 2 + 8 * kh, &r[3 * g]);
        else lds_dwords<2, true>(p + 18 * g + 2 + 8 * kh, &r[3 * g]);
        r[3 * g + 2] = at16(p + 18 * g);
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
    static constexpr bool OFF = true, EARLY = true;
    struct Pre { uint32_t m[4]; };
    __host__ __device__ static int kbase(int p) { return kbase_nibble(p); }
    __host__ __device__ static float xscale(int p) { return (p >> 1) & 1 ? 0.0625f : 1.0f; }
    __host__ __device__ static constexpr int step(int i) { return i; }
    static constexpr int LP = 5, ROW = 80;
    __device__ static uint32_t TB(int kt) { return 80u * (uint32_t)kt; }
    __device__ static uint32_t at(int j) { return 16u * (uint32_t)j; }
    __device__ static uint32_t odd(int) { return 0u; }
    __device__ static void read(const uint8_t *p, int kh, int g, uint32_t (&r)[NW]) {
        lds_dwords<2, false>(p + 20 * g + 4 + 8 * kh, &r[3 * g]);
        r[3 * g + 2] = at32(p + 20 * g);
    }
    __device__ static void prep(const uint32_t (&)[NW], int, int, Pre &) {}
    // also keeps the block's minimum: the four meet [S0 S2 S1 S3] hi and lo (lane half 0)
    __device__ static float scale(const uint32_t (&r)[NW], int st, int nb, Pre &p) {
        const int b = st >> 1;
        p.m[b] = b < nb ? r[3 * b + 2] >> 16 : 0u;
        return b < nb ? h2f(r[3 * b + 2]) : 0.f;
    }
    static constexpr bool PAIR = false;  // every k-tile; the minima stand for themselves (scale 1)
    __device__ static half8 offset(const uint8_t *, int, const Pre &p, float &) {
        const half2v a = h2(p.m[0] | (p.m[2] << 16)), c = h2(p.m[1] | (p.m[3] << 16));
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
    static constexpr bool OFF = false, EARLY = true;
    struct Pre {};
    __host__ __device__ static int kbase(int p) { return 32 * (p >> 2) + 16 * (p & 1) + 8 * ((p >> 1) & 1); }
    __host__ __device__ static float xscale(int) { return 1.0f; }
    __host__ __device__ static constexpr int step(int i) { return i; }
    static constexpr int LP = 9, ROW = 144;  // 136 bytes
    __device__ static uint32_t TB(int kt) { return 136u * (uint32_t)kt; }
    __device__ static uint32_t at(int j) { return 16u * (uint32_t)j; }
    __device__ static uint32_t odd(int) { return 0u; }
    __device__ static void read(const uint8_t *p, int kh, int g, uint32_t (&r)[NW]) {
        if (g & 1) lds_dwords<4, false>(p + 34 * g + 2 + 16 * kh, &r[5 * g]);
        else lds_dwords<4, true>(p + 34 * g + 2 + 16 * kh, &r[5 * g]);
        r[5 * g + 4] = at16(p + 34 * g);
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
// four 6-bit scales (or minima) of sub-blocks 4 t .. 4 t + 3, one per byte; t is
// 0 or ~0 (masks: a uniform branch per dword costs more than both sides)
__device__ __forceinline__ uint32_t k_scales4(uint32_t s0, uint32_t s2, uint32_t t) {
    return (s0 & 0x3F3F3F3Fu & ~t) | (((s2 & 0x0F0F0F0Fu) | ((s0 >> 2) & 0x30303030u)) & t);
}
__device__ __forceinline__ uint32_t k_mins4(uint32_t s1, uint32_t s2, uint32_t t) {
    return (s1 & 0x3F3F3F3Fu & ~t) | ((((s2 >> 4) & 0x0F0F0F0Fu) | ((s1 >> 2) & 0x30303030u)) & t);
}
template <int QH>
struct MDecK {
    static constexpr int NW = 12 + 4 * QH, STEPS = 8, NG = 2, BB = QH ? 176 : 144;
    static constexpr bool OFF = true, EARLY = false;
    struct Pre {
        half2v a, b;  // sc of sub-blocks (0, 2) times 2^10 and (1, 3) times 2^6
        float d;
    };
    __host__ __device__ static int kbase(int p) { return kbase_k(p); }
    __host__ __device__ static float xscale(int) { return 1.0f; }
    __host__ __device__ static constexpr int step(int i) { return i; }
    // pieces: the 64 code bytes of the half super-block, qh[32] (Q5_K), the header
    static constexpr int LP = QH ? 7 : 5, ROW = 16 * LP;
    __device__ static uint32_t TB(int kt) { return (uint32_t)BB * (uint32_t)(kt >> 1); }
    __device__ static uint32_t at(int j) { return j < 4 ? 16u + 32u * QH + 16u * (uint32_t)j : j < LP - 1 ? 16u * (uint32_t)(j - 3) : 0u; }
    __device__ static uint32_t odd(int j) { return j < 4 ? 64u : 0u; }
    __device__ static void read(const uint8_t *p, int kh, int g, uint32_t (&r)[NW]) {
        const u32x4_t q = at128(p + 32 * g + 16 * kh);
        r[4 + 4 * g] = q.x; r[5 + 4 * g] = q.y; r[6 + 4 * g] = q.z; r[7 + 4 * g] = q.w;
        if (g == 0) {
            const u32x4_t h = at128(p + ROW - 16);
            r[0] = h.x; r[1] = h.y; r[2] = h.z; r[3] = h.w;
            if constexpr (QH) {
                const u32x4_t b = at128(p + 64 + 16 * kh);
                r[NW - 4] = b.x; r[NW - 3] = b.y; r[NW - 2] = b.z; r[NW - 1] = b.w;
            }
        }
    }
    __device__ static void prep(const uint32_t (&r)[NW], int kt, int, Pre &p) {
        const uint32_t sc = k_scales4(r[1], r[3], (uint32_t)-(kt & 1));
        p.a = byte02_code(sc, 0.f) * splat(1024.f);
        p.b = byte13_code(sc, 0.f) * splat(64.f);
        p.d = h2f(r[0]) * 16384.f;
    }
    __device__ static float scale(const uint32_t (&)[NW], int, int, const Pre &p) { return p.d; }
    // the minima of the whole super-block in one step, after its second k-tile:
    // lane half kh holds those of k-tile kh
    static constexpr bool PAIR = true;
    __device__ static half8 offset(const uint8_t *p, int kh, const Pre &, float &so) {
        const u32x4_t h = at128(p + ROW - 16);  // the header again, from LDS: no registers held for it
        const uint32_t mn = k_mins4(h.z, h.w, (uint32_t)-kh);
        so = -h2f(h.x >> 16);
        const half2v m = byte02_code(mn, 0.f), n = byte13_code(mn, 0.f);  // [m0 m2], [m1 m3]
        return join(m, n, m, n);
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
    static constexpr bool OFF = false, EARLY = true;
    struct Pre { float d; };
    __host__ __device__ static constexpr int step(int i) { return 2 * (i & 3) + (i >> 2); }
    __host__ __device__ static int kbase(int p) { return 16 * step(p >> 1) + 8 * (p & 1); }
    __host__ __device__ static float xscale(int) { return 1.0f; }
    // pieces: ql[64] of the half, qh[32], its 8 sub-scales (and 8 bytes more), the
    // super-block's last 16 bytes, which d ends
    static constexpr int LP = 8, ROW = 144;
    __device__ static uint32_t TB(int kt) { return 210u * (uint32_t)(kt >> 1); }
    __device__ static uint32_t at(int j) { return j < 4 ? 16u * (uint32_t)j : j < 6 ? 64u + 16u * (uint32_t)j : j == 6 ? 192u : 194u; }
    __device__ static uint32_t odd(int j) { return j < 4 ? 64u : j < 6 ? 32u : j == 6 ? 8u : 0u; }
    __device__ static void read(const uint8_t *p, int kh, int g, uint32_t (&r)[NW]) {
        const u32x2_t a = at64(p + 16 * g + 8 * kh), b = at64(p + 32 + 16 * g + 8 * kh), c = at64(p + 64 + 16 * g + 8 * kh);
        r[6 * g] = a.x; r[6 * g + 1] = a.y; r[6 * g + 2] = b.x; r[6 * g + 3] = b.y; r[6 * g + 4] = c.x; r[6 * g + 5] = c.y;
        if (g == 0) {
            const u32x2_t sc = at64(p + 96);
            r[12] = sc.x; r[13] = sc.y;
            r[14] = at16(p + 126);
        }
    }
    __device__ static void prep(const uint32_t (&r)[NW], int, int, Pre &p) {
        p.d = h2f(r[14]);
    }
    __device__ static float scale(const uint32_t (&r)[NW], int st, int, const Pre &p) {
        return p.d * (float)(int)(int8_t)(uint8_t)(r[12 + (st >> 2)] >> (8 * (st & 3)));
    }
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
// The workspace of one call.  tiles[0].x = number of tiles; tile i is tiles[1 +
// i] = (expert, first position in order, rows | tiles of the expert << 8, first
// tile of the expert).
struct MoeWs {
    int4 *tiles;
    int32_t *order;   // the slots, expert after expert
    float *rscale;    // per row: what the split row was divided by
    uint4 *sums;      // [row][k-tile]: 4 block sums, hi and lo (formats with minima)
    uint8_t *xs;      // [row][half k-tile][hi, lo][8 pieces of 8 values]
    float *prod;      // down: [split][slot][M]; gate/up with splits: [split][slot][gate, up][M]
};

// Block 0 sorts the S slots by expert and cuts each expert's run into tiles of
// BN; the order of slots within an expert moves no result (every output row
// depends on its own activation row alone).
__device__ void plan_tiles(const int32_t *ids, int S, int E, int BN, int4 *tiles, int32_t *order) {
    __shared__ int count[MOE_E_MAX], start[MOE_E_MAX], tile0[MOE_E_MAX];
    const int t = (int)threadIdx.x, T = (int)blockDim.x;
    // the first slots' ids stay in registers between the two passes
    constexpr int KEEP = 16;
    int mine[KEEP];
#pragma unroll
    for (int i = 0; i < KEEP; i++) mine[i] = t + i * T < S ? ids[t + i * T] : -1;
    for (int e = t; e < E; e += T) count[e] = 0;
    __syncthreads();
    auto add = [&](int e) {
        if (e >= 0 && e < E) atomicAdd(&count[e], 1);
    };
#pragma unroll
    for (int i = 0; i < KEEP; i++) add(mine[i]);
    for (int s = t + KEEP * T; s < S; s += T) add(ids[s]);
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
        const int c = count[e], s0 = start[e], tc = (c + BN - 1) / BN;
        for (int i = 0; i < tc; i++)
            tiles[1 + tile0[e] + i] = int4{e, s0 + i * BN, (c - i * BN < BN ? c - i * BN : BN) | tc << 8, tile0[e]};
    }
    __syncthreads();
    auto put = [&](int s, int e) {
        if (e >= 0 && e < E) order[atomicAdd(&start[e], 1)] = s;
    };
#pragma unroll
    for (int i = 0; i < KEEP; i++) put(t + i * T, mine[i]);
    for (int s = t + KEEP * T; s < S; s += T) put(s, ids[s]);
}

// One piece (8 values, in the operand order) of a split row: 16 bytes of hi, 16 of lo.
template <int DT>
__device__ __forceinline__ void put_piece(const MoeWs &ws, int64_t row, int nkt, int i, const floatx4 &a, const floatx4 &b, float mul) {
    const int kt = i >> 4, p = i & 15;
    const float f = mul * MDec<DT>::xscale(p);
    const float v[8] = {a.x, a.z, a.y, a.w, b.x, b.z, b.y, b.w};
    half8 hi, lo;
    float sum = 0.f;
#pragma unroll
    for (int j = 0; j < 8; j++) {
        const float s = v[j] * f;
        sum += mul * v[j];
        hi[j] = (_Float16)s;
        const float r = s - (float)hi[j];
        lo[j] = (_Float16)(r == r ? r : 0.f);  // a non-finite x is in hi alone
    }
    half8 *o8 = reinterpret_cast<half8 *>(ws.xs + (row * nkt + kt) * (int64_t)KT_BYTES + (p >> 3) * XT_BYTES);
    o8[p & 7] = hi;
    o8[8 + (p & 7)] = lo;
    if constexpr (MDec<DT>::OFF) {
        // block b of the k-tile is pieces 4b .. 4b + 3: four neighbouring lanes
        sum += __shfl_xor(sum, 1, 64);
        sum += __shfl_xor(sum, 2, 64);
        const int l = (int)threadIdx.x & 48;
        const float s[4] = {__shfl(sum, l, 64), __shfl(sum, l + 8, 64), __shfl(sum, l + 4, 64), __shfl(sum, l + 12, 64)};
        if (p == 0) {
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

// Workgroup 0 plans the tiles; the others split rows, WPR of their 4 wavefronts
// on each.  PPL > 0: a row (K <= 512 WPR PPL) stays in registers between its
// maximum and the split, PPL pieces per lane; else it is read twice (1024 rows of
// 14336: 27 us read twice, 22.6 in registers).  zero_out (gate/up): the output rows [M]
// of a token's slots without an expert are cleared here, for the GEMM writes
// only rows that have one.  slot_rows (down): rows are slots, and those without
// an expert are skipped.
template <int DT, int WPR, int PPL>
__global__ void __launch_bounds__(256) moe_prep_kernel(const int32_t *ids, int S, int E, int BN, MoeWs ws, const float *X,
                                                       int64_t rows, int K, int nkt, int T, bool slot_rows, float *zero_out,
                                                       int64_t M) {
    if (blockIdx.x == 0) {
        plan_tiles(ids, S, E, BN, ws.tiles, ws.order);
        return;
    }
    __shared__ float red[4];
    constexpr int TPR = 64 * WPR;  // threads per row
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6), t = (int)threadIdx.x % TPR;
    const int64_t row = ((int64_t)blockIdx.x - 1) * (4 / WPR) + wave / WPR;
    const bool in = row < rows;
    bool live = in;
    if (in && slot_rows) {
        const int e = ids[row];
        live = e >= 0 && e < E;
    } else if (in) {
        for (int i = 0; i < T; i++) {
            const int e = ids[row * T + i];
            if (e < 0 || e >= E)
                for (int64_t m = t; m < M; m += TPR) zero_out[(row * T + i) * M + m] = 0.f;
        }
    }
    const int n = nkt * 16;  // pieces; lanes of a 16-lane group are in or out together
    const Rsrc rs = make_rsrc_uniform(X + (live ? row : 0) * K, live ? 4u * (uint32_t)K : 0u);  // zeros past the row
    float amax = 0.f;
    auto fold = [&](const floatx4 &v) {
#pragma unroll
        for (int j = 0; j < 4; j++) {
            const float a = fabsf(v[j]);
            amax = (a > amax && a < __builtin_inff()) ? a : amax;
        }
    };
    auto load = [&](int i, floatx4 &a, floatx4 &b) {
        const uint32_t k = 4u * (uint32_t)((i >> 4) * KT + MDec<DT>::kbase(i & 15));
        a = __builtin_bit_cast(floatx4, ld128(rs, k, 0));
        b = __builtin_bit_cast(floatx4, ld128(rs, k + 16u, 0));
    };
    floatx4 va[PPL > 0 ? PPL : 1], vb[PPL > 0 ? PPL : 1];
    if constexpr (PPL > 0) {
#pragma unroll
        for (int j = 0; j < PPL; j++) load(t + TPR * j, va[j], vb[j]);
#pragma unroll
        for (int j = 0; j < PPL; j++) { fold(va[j]); fold(vb[j]); }
    } else {
        for (int i = t; i < n; i += TPR) {
            load(i, va[0], vb[0]);
            fold(va[0]);
            fold(vb[0]);
        }
    }
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor(amax, o, 64));
    if constexpr (WPR > 1) {
        if ((threadIdx.x & 63) == 0) red[wave] = amax;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < WPR; w++) amax = fmaxf(amax, red[wave / WPR * WPR + w]);
    }
    if (!live) return;
    // amax = f * 2^e, f in [0.5, 1): multiply by 2^(10 - e)
    int e = 0;
    (void)frexpf(amax, &e);
    int m = amax > 0.f ? 10 - e : 0;
    m = m > 126 ? 126 : m;
    const float mul = ldexpf(1.0f, m);
    if (t == 0) ws.rscale[row] = ldexpf(1.0f, -m);
    if constexpr (PPL > 0) {
#pragma unroll
        for (int j = 0; j < PPL; j++)
            if (t + TPR * j < n) put_piece<DT>(ws, row, nkt, t + TPR * j, va[j], vb[j], mul);
    } else {
        for (int i = t; i < n; i += TPR) {
            load(i, va[0], vb[0]);
            put_piece<DT>(ws, row, nkt, i, va[0], vb[0], mul);
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
    int splits, kper;        // workgroups that share a row tile's K, k-tiles of each (even)
    int64_t part_stride;     // floats between the splits' parts in ws.prod
    uint32_t xs_bytes;       // of ws.xs
};

// k-tiles [k0, k1) of one job: W wavefronts, each 2 x 32 rows of the matrix
// (swiglu: 32 gate rows and the same 32 up rows) against the n_rows <= 32 FN
// slots of a tile.  Weights: a wavefront loads its own rows' bytes of a k-tile, 5
// to 9 lanes next to each other on a row (lanes reading a row each would touch
// 32 cache lines per instruction), parks them in its part of LDS one k-tile ahead and reads each
// lane's bytes from there.  Activations: all wavefronts share the tile's rows,
// double-buffered.
template <int DT, int FN, int BN, int W, bool SWI>
__device__ __forceinline__ void moe_tile(const MoeGemmArgs &a, const int4 tile, int e, int n_rows, int mt, int split, int k0, int k1,
                                         uint8_t (*xl)[BN * XT_BYTES], uint8_t (*wl)[WL_ROWS * MDec<DT>::ROW], int32_t *slot_of,
                                         float *rsc) {
    using D = MDec<DT>;
    constexpr int FR = 32 * FN, RW = SWI ? 32 : 64, BM = RW * W;
    constexpr int NP = FR * 16 / (64 * W);  // 16-byte pieces of half a k-tile per thread
    static_assert(NP >= 1, "tile too small for the workgroup");
    // rows per load instruction (lanes past them start the next row), instructions
    // per half (gate and up rows come from two blobs) and k-tile
    constexpr int RI = 64 / D::LP, HALVES = SWI ? 2 : 1, MH = (64 / HALVES + RI - 1) / RI, MI = HALVES * MH;
    constexpr int HROWS = (MH - 1) * RI + 63 / D::LP + 1;  // rows that a half's loads bring
    constexpr int HALF2 = SWI ? HROWS : 32;                // the second 32 rows' first in LDS
    static_assert(HALVES * HROWS <= WL_ROWS, "rows behind the last overrun the wavefront's LDS");
    const int t = (int)threadIdx.x, lane = t & 63, wave = __builtin_amdgcn_readfirstlane(t >> 6);
    const int l32 = lane & 31, kh = lane >> 5;
    for (int i = t; i < FR; i += 64 * W) {
        const int s = i < n_rows ? a.ws.order[tile.y + i] : -1;
        slot_of[i] = s;
        rsc[i] = s >= 0 ? a.ws.rscale[s / a.T] : 0.f;
    }
    __syncthreads();

    // activation pieces: piece c of thread t is 16-byte piece t % 16 of row t / 16 + c (4 W),
    // kept at piece (t % 16) ^ (row % 16) in LDS: 16 rows' reads of one piece
    // fall on 16 different bank groups
    static_assert((4 * W) % 16 == 0, "a thread's pieces lie in rows that agree modulo 16");
    uint32_t xoff[NP];
    const uint32_t xdst = (uint32_t)((t >> 4) * XT_BYTES + 16 * ((t ^ (t >> 4)) & 15));
#pragma unroll
    for (int c = 0; c < NP; c++) {
        const int r = (t >> 4) + c * (4 * W), p = t & 15;
        const int s = slot_of[r];
        // rows past the tile's end read nothing (zeros)
        xoff[c] = s >= 0 ? (uint32_t)(s / a.T) * (uint32_t)(a.nkt * KT_BYTES) + 16u * p : 0xFFFFFFF0u - (uint32_t)(a.nkt * KT_BYTES);
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
    const uint32_t rb = (uint32_t)a.row_bytes;
    const uint32_t so1 = SWI ? 0u : 32u * rb;   // the second 32 rows: of the up matrix, or further down
    const uint32_t moff = mis + (uint32_t)(lane / D::LP) * rb + D::at(lane % D::LP);
    const uint32_t modd = D::odd(lane % D::LP);
    uint8_t *const wmain = &wl[wave][(lane / D::LP) * D::ROW + 16 * (lane % D::LP)];
    uint8_t *const wrow[2] = {&wl[wave][l32 * D::ROW], &wl[wave][(HALF2 + l32) * D::ROW]};

    // block sums of the lane's slots (formats with minima): lane half 0 alone
    uint32_t sumoff[FN];
    const Rsrc srs = make_rsrc_uniform(a.ws.sums, D::OFF ? a.xs_bytes / (KT_BYTES / 16) : 0u);
    if constexpr (D::OFF) {
#pragma unroll
        for (int f = 0; f < FN; f++) {
            const int s = slot_of[32 * f + l32];
            sumoff[f] = 16u * ((uint32_t)(s >= 0 ? s / a.T : 0) * (uint32_t)a.nkt + (D::PAIR ? (uint32_t)kh : 0u));
        }
    }

    floatx16 acc[2][FN];
#pragma unroll
    for (int i = 0; i < 2; i++)
#pragma unroll
        for (int f = 0; f < FN; f++)
#pragma unroll
            for (int j = 0; j < 16; j++) acc[i][f][j] = 0.f;

    // Rows past a half's last are behind the resource's end (zeros) and have
    // their own place in LDS.
    u32x4_t wm[MI];
    auto fetch_w = [&](int kt) {
        const uint32_t tb = D::TB(kt), off = moff + (kt & 1 ? modd : 0u);
#pragma unroll
        for (int i = 0; i < MI; i++)
            wm[i] = ld128(i >= MH ? wr1 : wr0, off, tb + (uint32_t)(i % MH * RI) * rb);
    };
    // A row of 18- or 34-byte blocks may end inside a dword, which reads as 0
    // where it reaches past the matrix: its last two bytes are loaded by
    // themselves, once, and written over the last k-tile's (into the padding of
    // the others').
    constexpr bool TAIL = DT == QMM_Q4_0 || DT == QMM_Q8_0;
    uint32_t tail[2] = {0u, 0u};
    if constexpr (TAIL) {
        const uint32_t end = mis + (uint32_t)l32 * rb + rb - 2u;
        tail[0] = ld16(wr0, end, 0u);
        tail[1] = ld16(wr1, end + so1, 0u);
    }
    auto store_w = [&](int kt) {
#pragma unroll
        for (int i = 0; i < MI; i++) *reinterpret_cast<u32x4_t *>(wmain + (i / MH * HALF2 + i % MH * RI) * D::ROW) = wm[i];
        if constexpr (TAIL) {
            const int at = kt == a.nkt - 1 ? (int)rb - (int)D::TB(kt) - 2 : D::ROW - 4;
            *reinterpret_cast<uint16_t *>(wrow[0] + at) = (uint16_t)tail[0];
            *reinterpret_cast<uint16_t *>(wrow[1] + at) = (uint16_t)tail[1];
        }
    };
    uint32_t raw[2][D::NW];
    auto read_w = [&](int g) {
        D::read(wrow[0], kh, g, raw[0]);
        D::read(wrow[1], kh, g, raw[1]);
    };
    // A wavefront that has read all of its raw bytes puts the next k-tile's in
    // their place, which no other wavefront sees: under the last step's matrix
    // instructions (512 tokens, 14336 x 4096 Q6_K: 868 us against 889), but for
    // formats whose minima are read after it (Q5_K: 672 us, 715 with them kept in
    // registers).
    constexpr bool EARLY = D::EARLY;
    auto next_w = [&](int kn) {
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        store_w(kn);
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        read_w(0);
    };
    u32x4_t xr[NP];
    const int nx = 2 * k1;  // past the last half k-tile
    auto fetch_x = [&](int x) {  // past the last one: the last again, unused
#pragma unroll
        for (int c = 0; c < NP; c++) xr[c] = ld128(xrs, xoff[c], (uint32_t)((x < nx ? x : nx - 1) * XT_BYTES));
    };
    auto store_x = [&](int buf) {
#pragma unroll
        for (int c = 0; c < NP; c++) *reinterpret_cast<u32x4_t *>(&xl[buf][xdst + c * (4 * W) * XT_BYTES]) = xr[c];
    };
    fetch_x(2 * k0);
    fetch_w(k0);
    store_x(0);
    fetch_x(2 * k0 + 1);
    store_w(k0);
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    read_w(0);
    __syncthreads();

    for (int kt = k0; kt < k1; kt++) {
        const int kn = kt + 1 < k1 ? kt + 1 : kt;  // past the last k-tile: the last again, unused
        u32x4_t so_a[FN];
        const int nb = (a.K - kt * KT) / 32;
        typename D::Pre pre[2];
        floatx16 tmp[2][FN];
#pragma unroll
        for (int n = 0; n < 8; n++) {
            const int st = D::step(n), h = n >> 2;
            if (n % 4 == 0) {
                // half h of the k-tile: the other buffer takes the half after it
                // (fetched half a k-tile ago), and the one after that sets out
                store_x(h ^ 1);
                fetch_x(2 * kt + h + 2);
            }
            if constexpr (D::OFF) {
                // block sums for the step at the k-tile's (super-block's) end.
                // Loads return in order: asked for behind the next weights they
                // would wait for those (512 tokens, 14336 x 4096 Q4_K: 603 us
                // against 578)
                if (n == 0 && (!D::PAIR || (kt & 1))) {
#pragma unroll
                    for (int f = 0; f < FN; f++) so_a[f] = ld128(srs, sumoff[f], 16u * (uint32_t)(D::PAIR ? kt - 1 : kt));
                }
            }
            if (n == 0) {
                fetch_w(kn);
#pragma unroll
                for (int i = 0; i < 2; i++) D::prep(raw[i], kt, nb, pre[i]);
            }
            if (n % (8 / D::NG) == 0 && n / (8 / D::NG) + 1 < D::NG) read_w(n / (8 / D::NG) + 1);
            half8 b[2];
#pragma unroll
            for (int i = 0; i < 2; i++) b[i] = D::frag(raw[i], st, kt, pre[i]);
            float cs[2];  // the scale of the chain that this step ends
            if ((n + 1) % D::STEPS == 0) {
#pragma unroll
                for (int i = 0; i < 2; i++) cs[i] = D::scale(raw[i], st, nb, pre[i]);
            }
            if (EARLY && n == 7) next_w(kn);
            const uint8_t *xb = &xl[h][l32 * XT_BYTES];
            const int p = ((2 * (n & 3) + kh) ^ l32) & 15;
            half8 ah[FN], al[FN];
#pragma unroll
            for (int f = 0; f < FN; f++) {
                ah[f] = *reinterpret_cast<const half8 *>(xb + 32 * f * XT_BYTES + 16 * p);
                al[f] = *reinterpret_cast<const half8 *>(xb + 32 * f * XT_BYTES + 16 * (p ^ 8));
            }
#pragma unroll
            for (int f = 0; f < FN; f++)
#pragma unroll
                for (int i = 0; i < 2; i++) {
                    if (n % D::STEPS == 0) {
                        floatx16 z;
#pragma unroll
                        for (int j = 0; j < 16; j++) z[j] = 0.f;
                        tmp[i][f] = __builtin_amdgcn_mfma_f32_32x32x16_f16(al[f], b[i], z, 0, 0, 0);
                    } else {
                        tmp[i][f] = __builtin_amdgcn_mfma_f32_32x32x16_f16(al[f], b[i], tmp[i][f], 0, 0, 0);
                    }
                }
#pragma unroll
            for (int f = 0; f < FN; f++)
#pragma unroll
                for (int i = 0; i < 2; i++) tmp[i][f] = __builtin_amdgcn_mfma_f32_32x32x16_f16(ah[f], b[i], tmp[i][f], 0, 0, 0);
            if ((n + 1) % D::STEPS == 0) {
                // the end of a chain: scale its sum once, in f32
#pragma unroll
                for (int i = 0; i < 2; i++) {
#pragma unroll
                    for (int f = 0; f < FN; f++)
#pragma unroll
                        for (int j = 0; j < 16; j++) acc[i][f][j] = fmaf(cs[i], tmp[i][f][j], acc[i][f][j]);
                }
            }
            if (n == 3) __syncthreads();
            // one chain's sums at a time: left alone the compiler starts
            // several and spills them
            else if ((n + 1) % D::STEPS == 0) __builtin_amdgcn_sched_barrier(0);
        }
        if constexpr (D::OFF) {
            if (!D::PAIR || (kt & 1)) {
                float so[2];
                half8 off[2], sa[FN];
#pragma unroll
                for (int f = 0; f < FN; f++)
                    sa[f] = D::PAIR || kh == 0 ? __builtin_bit_cast(half8, so_a[f]) : half8{0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll
                for (int i = 0; i < 2; i++) off[i] = D::offset(wrow[i], kh, pre[i], so[i]);
#pragma unroll
                for (int f = 0; f < FN; f++)
#pragma unroll
                    for (int i = 0; i < 2; i++) {
                        if constexpr (D::PAIR) {
                            floatx16 z;
#pragma unroll
                            for (int j = 0; j < 16; j++) z[j] = 0.f;
                            tmp[i][f] = __builtin_amdgcn_mfma_f32_32x32x16_f16(sa[f], off[i], z, 0, 0, 0);
                        } else {
                            acc[i][f] = __builtin_amdgcn_mfma_f32_32x32x16_f16(sa[f], off[i], acc[i][f], 0, 0, 0);
                        }
                    }
                if constexpr (D::PAIR) {
                    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                    for (int f = 0; f < FN; f++)
#pragma unroll
                        for (int i = 0; i < 2; i++)
#pragma unroll
                            for (int j = 0; j < 16; j++) acc[i][f][j] = fmaf(so[i], tmp[i][f][j], acc[i][f][j]);
                }
            }
        }
        if (!EARLY) next_w(kn);
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
                const float v0 = acc[0][f][j] * sc, v1 = acc[1][f][j] * sc;
                if (SWI && a.splits == 1) {
                    if (l32 < left) a.out[s * a.M + m0 + l32] = silu(v0) * v1;
                } else if (SWI) {
                    float *o = a.ws.prod + split * a.part_stride + 2 * s * a.M + m0 + l32;
                    if (l32 < left) { o[0] = v0; o[a.M] = v1; }
                } else {
                    float *o = a.ws.prod + split * a.part_stride + s * a.M + m0 + l32;
                    if (l32 < left) o[0] = v0;
                    if (l32 + 32 < left) o[32] = v1;
                }
            }
        }
}

// Registers: with two wavefronts per SIMD a lane has 256.  Tiles of 32 slots take
// 153-194, tiles of 64 239-255, but for Q4_1 and Q6_K, which need 5 to 9 more and keep
// those in scratch memory (24-40 bytes a lane): 512 tokens of 14336 x 4096 write 68
// and 121 MB where the outputs are 59.
//
// One workgroup per job.  A tile of 64 that holds up to 32 slots, often an
// expert's last one, runs half of the matrix steps (down of 2 of 8 experts 4096 x
// 14336 Q6_K, 512 tokens: 685 us against 728 with every tile run in full; of 8 of
// 64 experts 4096 x 1024 Q8_0: 187 against 195).
template <int DT, int FN, int W, bool SWI>
__global__ void __launch_bounds__(64 * W, 2) moe_gemm_kernel(const MoeGemmArgs a) {
    constexpr int BN = 32 * FN;
    __shared__ __attribute__((aligned(16))) uint8_t xl[2][BN * XT_BYTES];           // two half k-tiles of activations
    __shared__ __attribute__((aligned(16))) uint8_t wl[W][WL_ROWS * MDec<DT>::ROW];  // each wavefront's rows
    __shared__ int32_t slot_of[BN];
    __shared__ float rsc[BN];
    // An XCD (workgroup id mod 8) takes a run of jobs, ordered by expert, then
    // rows of its matrix, then its tiles of slots: the workgroups running on it
    // at a time share one expert's slots (a few MB, its L2) and read the same
    // rows together
    const int per_tile = a.mtiles * a.splits;
    const int nt = a.ws.tiles[0].x, total = nt * per_tile, chunk = (total + 7) / 8;
    const int id = ((int)blockIdx.x & 7) * chunk + ((int)blockIdx.x >> 3);
    if (((int)blockIdx.x >> 3) >= chunk || id >= total) return;
    const int4 of_job = a.ws.tiles[1 + id / per_tile];  // some tile of the job's expert
    const int t0 = of_job.w, tc = of_job.z >> 8, r_id = id - t0 * per_tile;
    const int mt = r_id / tc / a.splits, split = r_id / tc % a.splits;
    const int k0 = split * a.kper, k1 = k0 + a.kper < a.nkt ? k0 + a.kper : a.nkt;  // k-tiles [k0, k1)
    const int4 tile = a.ws.tiles[1 + t0 + r_id % tc];
    const int e = __builtin_amdgcn_readfirstlane(tile.x), n_rows = __builtin_amdgcn_readfirstlane(tile.z & 0xFF);
    if (FN == 1 || n_rows > 32) moe_tile<DT, FN, BN, W, SWI>(a, tile, e, n_rows, mt, split, k0, k1, xl, wl, slot_of, rsc);
    else moe_tile<DT, 1, BN, W, SWI>(a, tile, e, n_rows, mt, split, k0, k1, xl, wl, slot_of, rsc);
}

// Y[n][m] = residual[n][m] + sum over t of weights[n][t] * prod[n T + t][m], t
// ascending, a slot's product the sum of its splits' parts.  V values per thread (4: M % 4 == 0 and 16-byte aligned rows).
// Four slots' rows are in flight at once; a slot without an expert is an empty
// resource (zeros) under weight 0.
template <int V>
__global__ void __launch_bounds__(256) moe_combine_kernel(const int32_t *ids, const float *weights, const float *prod,
                                                          const float *residual, float *Y, int E, int64_t M, int T,
                                                          int splits, int64_t part_stride) {
    const int64_t n = blockIdx.x;
    const uint32_t bytes = 4u * (uint32_t)M;
    const Rsrc rr = make_rsrc_uniform(residual ? residual + n * M : prod, residual ? bytes : 0u);
    const Rsrc ry = make_rsrc_uniform(Y + n * M, bytes);
    for (uint32_t off = 4u * V * (blockIdx.y * 256u + threadIdx.x); off < bytes; off += 4u * V * 256u * gridDim.y) {
        float y[V];
        auto get = [&](Rsrc rs, float (&v)[V]) {
            if constexpr (V == 4) {
                const floatx4 q = __builtin_bit_cast(floatx4, ld128(rs, off, 0));
                v[0] = q.x; v[1] = q.y; v[2] = q.z; v[3] = q.w;
            } else {
                v[0] = __builtin_bit_cast(float, ld32(rs, off, 0));
            }
        };
        get(rr, y);
        for (int t0 = 0; t0 < T; t0 += 4) {
            float v[4][V], w[4];
#pragma unroll
            for (int j = 0; j < 4; j++) {
                const int64_t s = n * T + (t0 + j < T ? t0 + j : T - 1);
                const int e = ids[s];
                const bool live = t0 + j < T && e >= 0 && e < E;
                w[j] = live ? weights[s] : 0.f;
                get(make_rsrc_uniform(prod + s * M, live ? bytes : 0u), v[j]);
                for (int p = 1; p < splits; p++) {
                    float u[V];
                    get(make_rsrc_uniform(prod + p * part_stride + s * M, live ? bytes : 0u), u);
#pragma unroll
                    for (int i = 0; i < V; i++) v[j][i] += u[i];
                }
            }
#pragma unroll
            for (int j = 0; j < 4; j++)
#pragma unroll
                for (int i = 0; i < V; i++) y[i] = fmaf(w[j], v[j][i], y[i]);
        }
        if constexpr (V == 4)
            __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4_t, floatx4{y[0], y[1], y[2], y[3]}), ry, off, 0, 0);
        else
            __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(uint32_t, y[0]), ry, off, 0, 0);
    }
}

// out[slot][m] = silu(sum of the splits' gate parts) * (sum of their up parts)
__global__ void __launch_bounds__(256) moe_silu_parts_kernel(const int32_t *ids, const float *prod, float *out, int E, int64_t M,
                                                             int splits, int64_t part_stride) {
    const int64_t s = blockIdx.x;
    const int e = ids[s];
    if (e < 0 || e >= E) return;  // already cleared
    for (int64_t m = (int64_t)blockIdx.y * 256 + threadIdx.x; m < M; m += (int64_t)gridDim.y * 256) {
        float g = 0.f, u = 0.f;
        for (int p = 0; p < splits; p++) {
            g += prod[p * part_stride + 2 * s * M + m];
            u += prod[p * part_stride + (2 * s + 1) * M + m];
        }
        out[s * M + m] = silu(g) * u;
    }
}

// --------------------------------------------------------------- launchers ----
constexpr int64_t align256(int64_t v) { return (v + 255) & ~(int64_t)255; }

// Tokens per pass: the split rows and the down products stay below 1 GB (32-bit
// offsets), the grids below 2^32 threads; longer inputs run pass after pass in
// one workspace.
int64_t chunk_tokens(int64_t E, int64_t K, int64_t M, int64_t N, int64_t T, bool down) {
    const int64_t nkt = (K + KT - 1) / KT, row = nkt * KT_BYTES, mt = M / 128 + 1;
    int64_t n = (int64_t(1) << 30) / (down ? row * T : row);
    if (down) n = std::min(n, (int64_t(1) << 30) / (4 * M * T));
    n = std::min(n, (int64_t(1) << 22) / T);
    // (tiles of slots: slots / 32 and one per expert with any) x (row tiles) <= 2^23
    n = std::min(n, E * mt <= (int64_t(1) << 22) ? (int64_t(1) << 27) / (T * mt) : (int64_t(1) << 23) / (T * mt));
    return std::max<int64_t>(1, std::min(n, N));
}

constexpr int GEMM_W = 4;  // wavefronts per workgroup

// Slots per tile: 32 while an expert sees few of them, else 64 (half the weight
// reads and decoding per slot, but fewer and fuller workgroups).  64 experts, 8
// each, gate/up 1024 x 2048 Q4_K, tiles of 32 against 64: 200 tokens 83 against
// 102 us, 400 tokens (50 slots each) 114 against 125, 1000 tokens 209 against 200;
// down 2048 x 1024 Q8_0: 200 tokens 76 against 84, 400 tokens 101 against 95; 8
// experts, 2 each, 14336 x 4096 Q4_K: 192 tokens (48 slots) 325 against 344, 256
// tokens 410 against 395.
int moe_gemm_bn(int64_t E, int64_t N, int64_t T) { return N * T <= 48 * E ? 32 : 64; }

struct MoeSizes {
    int64_t tokens, slots, rows, nkt, tiles, mtiles, splits, kper;
    int64_t o_order, o_rscale, o_sums, o_xs, o_prod, bytes;
};
MoeSizes moe_sizes(int dtype, int64_t E, int64_t M, int64_t K, int64_t N, int64_t T, int BN, bool down) {
    MoeSizes z;
    z.tokens = chunk_tokens(E, K, M, N, T, down);
    z.slots = z.tokens * T;
    z.rows = down ? z.slots : z.tokens;
    z.nkt = (K + KT - 1) / KT;
    z.tiles = z.slots / BN + std::min(E, z.slots);
    z.mtiles = (M + (down ? 64 : 32) * GEMM_W - 1) / ((down ? 64 : 32) * GEMM_W);
    // Few jobs (a workgroup alone on its CU needs ~2 us per k-tile): the k-tiles
    // of a row tile are shared out, at least 8 each, until two workgroups per CU
    // have one.  Two wide experts' down projection, 30 tokens, 8 x 4096 x 14336
    // Q4_K: 253 us in one piece.
    const int64_t jobs = std::max<int64_t>(1, std::min(z.tiles, std::min(E, z.slots) + z.slots / (2 * BN)) * z.mtiles);
    z.splits = std::max<int64_t>(1, std::min<int64_t>({512 / jobs, z.nkt / 8, 8}));
    z.kper = ((z.nkt + z.splits - 1) / z.splits + 1) / 2 * 2;
    z.splits = (z.nkt + z.kper - 1) / z.kper;
    const bool off = dtype == QMM_Q4_1 || dtype == QMM_Q4_K || dtype == QMM_Q5_K;
    z.o_order = align256(16 * (1 + z.tiles));
    z.o_rscale = z.o_order + align256(4 * z.slots);
    z.o_sums = z.o_rscale + align256(4 * z.rows);
    z.o_xs = z.o_sums + (off ? align256(16 * z.rows * z.nkt) : 0);
    z.o_prod = z.o_xs + align256(z.rows * z.nkt * KT_BYTES);
    z.bytes = z.o_prod + (down ? align256(4 * z.splits * z.slots * M) : z.splits > 1 ? align256(8 * z.splits * z.slots * M) : 0);
    return z;
}

template <int DT, int FN, int W, bool SWI>
void launch_gemm(const MoeGemmArgs &a, int64_t tiles, hipStream_t st) {
    const int64_t blocks = (tiles * a.mtiles * a.splits + 7) / 8 * 8;
    hipLaunchKernelGGL((moe_gemm_kernel<DT, FN, W, SWI>), dim3((unsigned)blocks), dim3(64 * W), 0, st, a);
}

template <int DT, bool SWI>
hipError_t run_gemm(const void *w0, const void *w1, int64_t E, int64_t M, int64_t K, int64_t N, int64_t T, const int32_t *ids,
                    const float *weights, const float *X, const float *residual, float *out, void *work, hipStream_t st) {
    constexpr int W = GEMM_W;
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
    a.mtiles = (int)z.mtiles;
    a.splits = (int)z.splits;
    a.kper = (int)z.kper;
    a.T = SWI ? (int)T : 1;
    for (int64_t n0 = 0; n0 < N; n0 += z.tokens) {
        const int64_t n = std::min(z.tokens, N - n0), S = n * T, rows = SWI ? n : S;
        const int32_t *idc = ids + n0 * T;
        a.xs_bytes = (uint32_t)(rows * z.nkt * KT_BYTES);
        a.out = SWI ? out + n0 * T * M : nullptr;
        a.part_stride = (SWI ? 2 : 1) * S * M;
        const float *xc = X + n0 * (SWI ? 1 : T) * K;
        const int wpr = K <= 1024 ? 1 : K <= 2048 ? 2 : 4;  // wavefronts per row
        const dim3 pg((unsigned)((rows * wpr + 3) / 4 + 1));
#define QMM_PREP(WPR, PPL)                                                                                              \
    hipLaunchKernelGGL((moe_prep_kernel<DT, WPR, PPL>), pg, dim3(256), 0, st, idc, (int)S, (int)E, BN, a.ws, xc, rows, (int)K, \
                       (int)z.nkt, (int)T, !SWI, a.out, M)
        if (wpr == 1) QMM_PREP(1, 2);
        else if (wpr == 2) QMM_PREP(2, 2);
        else if (K <= 4096) QMM_PREP(4, 2);
        else if (K <= 8192) QMM_PREP(4, 4);
        else if (K <= 16384) QMM_PREP(4, 8);
        else QMM_PREP(4, 0);
#undef QMM_PREP
        const int64_t tiles = S / BN + std::min(E, S);
        if (BN == 32) launch_gemm<DT, 1, W, SWI>(a, tiles, st);
        else launch_gemm<DT, 2, W, SWI>(a, tiles, st);
        if (SWI && a.splits > 1) {
            const dim3 sg((unsigned)S, (unsigned)std::min<int64_t>((M + 255) / 256, 64));
            hipLaunchKernelGGL(moe_silu_parts_kernel, sg, dim3(256), 0, st, idc, a.ws.prod, a.out, (int)E, M, a.splits, a.part_stride);
        }
        if (!SWI) {
            const float *res = residual ? residual + n0 * M : nullptr;
            float *y = out + n0 * M;
            const bool vec = M % 4 == 0 && ((uintptr_t)res & 15) == 0 && ((uintptr_t)y & 15) == 0;
            const int64_t per = vec ? 1024 : 256;
            const dim3 cg((unsigned)n, (unsigned)std::min<int64_t>((M + per - 1) / per, 64));
            if (vec) hipLaunchKernelGGL((moe_combine_kernel<4>), cg, dim3(256), 0, st, idc, weights + n0 * T, a.ws.prod, res, y, (int)E, M, (int)T, a.splits, a.part_stride);
            else hipLaunchKernelGGL((moe_combine_kernel<1>), cg, dim3(256), 0, st, idc, weights + n0 * T, a.ws.prod, res, y, (int)E, M, (int)T, a.splits, a.part_stride);
        }
    }
    return hipGetLastError();
}

}  // namespace

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
