// qmm_rope.hip -- rotary positions and the cache append (include/qmm.h,
// qmm_rope, qmm_rope_freqs, qmm_kv_append).
//
// A pair (u, w) of a head at position pos turns by a = pos * f_i:
//     (u cos a - w sin a, u sin a + w cos a) * mscale
// The angle, its sine and cosine and the products are f64, and a result is
// rounded to f32 once: at position 2^17 an f32 angle is off by 2^-8 of a turn's
// radian, and the Q8_0 codes of a key next to a rounding border would hang on the
// last bits otherwise.  One sine and cosine per (token, pair) serves all heads of a
// workgroup through LDS.
//
// Bound by memory (one read, one write; about 6 f64 operations a pair): 4096 tokens of 40
// heads of 128 take 33 us, 5.1 TB/s, the rate of a large copy; one token of 32 heads 3.0 us, of
// which a launch is about 2.  Appending 4096 tokens of 32/8 heads to f16 pages takes 42 to 44 us
// (185 MB, 4.2 to 4.4 TB/s), to Q8_0 pages 3 more (177 MB).  A workgroup takes one token and up to 256 units of 8 values (for halves, 4
// neighbours of either half), one per thread, so that the loads are under way
// while a wavefront works out the angles.
//
// The append's values go to pages with the token index inside, so a workgroup
// takes TS neighbouring token places of 64 dims of a head: rows in, through LDS,
// places out, 16 bytes (8 places) a thread where all 8 are new.  (17 KB of LDS: whole
// heads of 128, 34 KB, halve the wavefronts of the turning workgroups in the same launch.)
#include "qmm_internal.hpp"
#include "qmm_kv.hpp"
#include "qmm_units.hpp"

namespace qmm {

namespace {

struct TurnArgs {
    const float *q, *k, *v;
    float *q_out;
    int64_t q_stride, k_stride, v_stride, out_stride;
    const int32_t *pos;
    const float *freqs, *q_norm, *k_norm;
    double mscale, eps;
    int Hq, Hk, D, rot, hpb, bpt;  // heads a workgroup, workgroups a token
    bool half;
    int64_t row0;                  // of a launch
    int64_t turn_blocks, v0, v_tiles;
    KvArgs kv;
};

// f32 -> Q8_0 code of one value, as q8_codes4 makes it
__device__ __forceinline__ int q8_code(float v, float id) {
    const float q = rintf(v * id);
    return (int)(q != q ? 0.0f : fminf(fmaxf(q, -128.0f), 127.0f));
}

// The values of 64 dims (or the last 32) of one head in TS neighbouring places (index
// t0 .. t0 + TS - 1).
constexpr int kDims = 64, kPitch = kDims + 1;
template <int DT, int TS>
__device__ __forceinline__ void put_values(const TurnArgs &a, int64_t vb, float *tile) {
    const KvArgs &kv = a.kv;
    const int t = (int)threadIdx.x, D = a.D, parts = (D + kDims - 1) / kDims;
    const uint32_t heads = (uint32_t)(a.Hk * parts);
    int h, s, k;
    if (a.v_tiles * kv.seqs * heads <= UINT32_MAX) {  // uniform
        const uint32_t b = (uint32_t)vb;
        h = (int)(b % heads);
        s = (int)(b / heads % (uint32_t)kv.seqs);
        k = (int)(b / heads / (uint32_t)kv.seqs);
    } else {
        h = (int)(vb % heads);
        s = (int)(vb / heads % kv.seqs);
        k = (int)(vb / heads / kv.seqs);
    }
    const int first = h % parts * kDims, W = D - first < kDims ? D - first : kDims;
    h /= parts;
    const KvNew nw = kv_new(kv, s);
    if (nw.count == 0 || nw.index + nw.count <= 0) return;
    const int64_t lo = nw.index > 0 ? nw.index : 0, hi = nw.index + nw.count;  // places lo .. hi - 1 are new
    const int64_t t0 = (lo / TS + k) * TS;
    if (t0 >= hi) return;
    const float *src = a.v + (int64_t)h * D + first;
    float x[TS * kDims / 256];
#pragma unroll
    for (int i = 0; i < TS * kDims / 256; i++) {  // all loads under way at once
        const int e = t + 256 * i, d = e % kDims;
        const int64_t at = t0 + e / kDims;
        x[i] = at >= lo && at < hi && d < W ? src[((int64_t)nw.first + (at - nw.index)) * a.v_stride + d] : 0.f;
    }
#pragma unroll
    for (int i = 0; i < TS * kDims / 256; i++) {
        const int e = t + 256 * i;
        tile[e / kDims * kPitch + e % kDims] = x[i];
    }
    __syncthreads();
    const int page = 1 << kv.page_shift, nb = W / 32;
    const int64_t rec = kv_record(DT, page, D);
    float *inv = tile + TS * kPitch;  // Q8_0: 1/d of [block][place]
    if constexpr (DT == QMM_Q8_0) {
        for (int e = t; e < TS * nb; e += 256) {
            const int j = e % TS, b = e / TS;
            const int64_t i = t0 + j;
            if (i < lo || i >= hi) continue;
            float amax = 0.f, d, id;
#pragma unroll 8
            for (int c = 0; c < 32; c++) {
                const float y = fabsf(tile[j * kPitch + 32 * b + c]);
                amax = y > amax ? y : amax;  // a NaN never wins
            }
            q8_scale(amax, d, id);
            inv[e] = id;
            const int pg = kv_page(kv, s, i);
            if (pg >= 0) {
                _Float16 *sc = reinterpret_cast<_Float16 *>(kv.v + ((int64_t)pg * kv.heads + h) * rec + (int64_t)page * D);
                sc[(first / 32 + b) * page + (int)(i & (page - 1))] = (_Float16)d;
            }
        }
        __syncthreads();
    }
    for (int e = t; e < W * (TS / 8); e += 256) {
        const int g = e % (TS / 8), d = e / (TS / 8);
        const int64_t i = t0 + 8 * g;
        if (i + 8 <= lo || i >= hi) continue;
        const int pg = kv_page(kv, s, i);  // 8 neighbours share a page
        if (pg < 0) continue;
        uint8_t *r = kv.v + ((int64_t)pg * kv.heads + h) * rec;
        const int at = (first + d) * page + (int)(i & (page - 1));
        const bool whole = i >= lo && i + 8 <= hi;
        const float *from = tile + 8 * g * kPitch + d;
        if constexpr (DT == QMM_F16) {
            _Float16 *o = reinterpret_cast<_Float16 *>(r) + at;
            half8 w;
#pragma unroll
            for (int j = 0; j < 8; j++) w[j] = (_Float16)from[j * kPitch];
            if (whole) {
                *reinterpret_cast<half8 *>(o) = w;
            } else {
#pragma unroll
                for (int j = 0; j < 8; j++)
                    if (i + j >= lo && i + j < hi) o[j] = w[j];
            }
        } else {
            int8_t *o = reinterpret_cast<int8_t *>(r) + at;
            uint32_t w[2] = {0u, 0u};
#pragma unroll
            for (int j = 0; j < 8; j++)
                w[j / 4] |= ((uint32_t)q8_code(from[j * kPitch], inv[(d / 32) * TS + 8 * g + j]) & 0xFFu) << (8 * (j % 4));
            if (whole) {
                *reinterpret_cast<u32x2_t *>(o) = u32x2_t{w[0], w[1]};
            } else {
#pragma unroll
                for (int j = 0; j < 8; j++)
                    if (i + j >= lo && i + j < hi) o[j] = (int8_t)(w[j / 4] >> (8 * (j % 4)));
            }
        }
    }
}

// DT 0: qmm_rope (queries only, positions by row).  Dynamic LDS: the V tile, or
// cos/sin of the pairs [rot/2], then the norms' partial sums [256], then the
// Q8_0 keys [256 * 8].
template <int DT, int TS>
__global__ void __launch_bounds__(256) turn_kernel(const TurnArgs a) {
    extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
    if constexpr (DT != 0) {
        if ((int64_t)blockIdx.x >= a.turn_blocks) {
            put_values<DT, TS>(a, a.v0 + ((int64_t)blockIdx.x - a.turn_blocks), reinterpret_cast<float *>(lds));
            return;
        }
    }
    const int t = (int)threadIdx.x;
    const uint32_t tok = blockIdx.x / (uint32_t)a.bpt;
    const int64_t n = a.row0 + tok;
    const int h0 = (int)(blockIdx.x - tok * (uint32_t)a.bpt) * a.hpb, H = a.Hq + a.Hk, D = a.D, uph = D / 8;
    int s = 0;
    int64_t index = 0;
    if constexpr (DT != 0) {
        s = kv_row_seq(a.kv, (int)n);
        if (s < 0) return;
        const KvNew nw = kv_new(a.kv, s);
        if (n - nw.first >= nw.count) return;
        index = nw.index + (n - nw.first);
    }
    const int hl = t / uph, u = t - hl * uph, head = h0 + hl;
    const bool on = hl < a.hpb && head < H, key = head >= a.Hq;
    // the unit's two groups of four values: dims d0 .. d0+3 and d1 .. d1+3
    const bool turned = 8 * u < a.rot;
    const int d0 = a.half && turned ? 4 * u : 8 * u, d1 = a.half && turned ? a.rot / 2 + 4 * u : 8 * u + 4;
    floatx4 x0{}, x1{}, w0{}, w1{};
    const float *norm = key ? a.k_norm : a.q_norm;
    if (on) {
        const float *src = key ? a.k + n * a.k_stride + (int64_t)(head - a.Hq) * D : a.q + n * a.q_stride + (int64_t)head * D;
        x0 = *reinterpret_cast<const floatx4 *>(src + d0);
        x1 = *reinterpret_cast<const floatx4 *>(src + d1);
        if (norm) {
            w0 = *reinterpret_cast<const floatx4 *>(norm + d0);
            w1 = *reinterpret_cast<const floatx4 *>(norm + d1);
        }
    }
    double2 *cs = reinterpret_cast<double2 *>(lds);
    double *part = reinterpret_cast<double *>(cs + a.rot / 2);
    const int64_t pos = a.pos ? (int64_t)a.pos[n] : index;
    for (int i = t; i < a.rot / 2; i += (int)blockDim.x) {
        double sn, cn;
        sincos((double)pos * (double)a.freqs[i], &sn, &cn);
        cs[i] = make_double2(cn * a.mscale, sn * a.mscale);
    }
    const bool norms = a.q_norm || a.k_norm;  // uniform
    if (norms) {
        double ss = 0.0;
#pragma unroll
        for (int j = 0; j < 4; j++) ss = fma((double)x0[j], (double)x0[j], fma((double)x1[j], (double)x1[j], ss));
        part[t] = ss;
    }
    __syncthreads();
    double y0[4], y1[4];
    double inv = 1.0;
    if (on && norm) {
        double ss = 0.0;
        for (int i = 0; i < uph; i++) ss += part[hl * uph + i];
        inv = 1.0 / sqrt(ss / D + a.eps);
    }
#pragma unroll
    for (int j = 0; j < 4; j++) {
        y0[j] = norm ? (double)x0[j] * inv * (double)w0[j] : (double)x0[j];
        y1[j] = norm ? (double)x1[j] * inv * (double)w1[j] : (double)x1[j];
    }
    if (turned) {
        if (a.half) {
#pragma unroll
            for (int j = 0; j < 4; j++) {
                const double2 c = cs[4 * u + j];
                const double p = y0[j], q = y1[j];
                y0[j] = fma(p, c.x, -(q * c.y));
                y1[j] = fma(p, c.y, q * c.x);
            }
        } else {
#pragma unroll
            for (int j = 0; j < 4; j += 2) {
                const double2 c = cs[4 * u + j / 2], e = cs[4 * u + 2 + j / 2];
                const double p = y0[j], q = y0[j + 1], r = y1[j], v = y1[j + 1];
                y0[j] = fma(p, c.x, -(q * c.y));
                y0[j + 1] = fma(p, c.y, q * c.x);
                y1[j] = fma(r, e.x, -(v * e.y));
                y1[j + 1] = fma(r, e.y, v * e.x);
            }
        }
    }
#pragma unroll
    for (int j = 0; j < 4; j++) {
        x0[j] = (float)y0[j];
        x1[j] = (float)y1[j];
    }
    if (on && !key) {
        float *o = a.q_out + n * a.out_stride + (int64_t)head * D;
        *reinterpret_cast<floatx4 *>(o + d0) = x0;
        *reinterpret_cast<floatx4 *>(o + d1) = x1;
    }
    if constexpr (DT == 0) return;
    if (h0 + a.hpb <= a.Hq) return;  // uniform: no keys here
    const KvArgs &kv = a.kv;
    const int pg = kv_page(kv, s, index);
    if (pg < 0) return;  // uniform
    const int page = 1 << kv.page_shift, place = (int)(index & (page - 1));
    const int64_t rec = kv_record(DT, page, D);
    if constexpr (DT == QMM_F16) {
        if (on && key) {
            _Float16 *o = reinterpret_cast<_Float16 *>(kv.k + ((int64_t)pg * kv.heads + (head - a.Hq)) * rec) + place * D;
            half4 g0, g1;
#pragma unroll
            for (int j = 0; j < 4; j++) {
                g0[j] = (_Float16)x0[j];
                g1[j] = (_Float16)x1[j];
            }
            *reinterpret_cast<half4 *>(o + d0) = g0;
            *reinterpret_cast<half4 *>(o + d1) = g1;
        }
    } else if constexpr (DT == QMM_Q8_0) {
        float *buf = reinterpret_cast<float *>(part + 256);
        if (hl < a.hpb) {
            *reinterpret_cast<floatx4 *>(buf + hl * D + d0) = x0;
            *reinterpret_cast<floatx4 *>(buf + hl * D + d1) = x1;
        }
        __syncthreads();
        // four neighbouring values a lane, eight lanes a block; 2 * 256 groups at most
#pragma unroll
        for (int r = 0; r < 2; r++) {
            const int e = t + 256 * r, l = e / (D / 4), d = 4 * (e - l * (D / 4)), hd = h0 + l;
            const bool in = l < a.hpb && hd < H && hd >= a.Hq;
            floatx4 v{};
            if (in) v = *reinterpret_cast<const floatx4 *>(buf + l * D + d);
            float sc;
            const uint32_t codes = q8_quant4(v, &sc);
            if (in) {
                uint8_t *o = kv.k + ((int64_t)pg * kv.heads + (hd - a.Hq)) * rec;
                *reinterpret_cast<uint32_t *>(o + place * D + d) = codes;
                if ((d & 31) == 0) reinterpret_cast<_Float16 *>(o + (int64_t)page * D)[(d / 32) * page + place] = (_Float16)sc;
            }
        }
    }
}

__global__ void __launch_bounds__(512) freqs_kernel(int rot, double base, double factor, double context, double fast,
                                                    double slow, const float *factors, float *freqs) {
    const int i = (int)threadIdx.x;
    if (i >= rot / 2) return;
    double f = pow(base, -2.0 * i / rot);
    if (factors) f /= (double)factors[i];
    double g = 1.0;  // the share of the stretched frequency
    if (context > 0.0) {
        const double two_pi = 6.283185307179586476925, den = 2.0 * log(base);
        const double low = fmax(floor(rot * log(context / (two_pi * fast)) / den), 0.0);
        const double high = fmin(ceil(rot * log(context / (two_pi * slow)) / den), (double)(rot - 1));
        g = fmin(fmax((i - low) / fmax(high - low, 0.001), 0.0), 1.0);
    }
    freqs[i] = (float)(f * (1.0 - g) + f / factor * g);
}

constexpr int64_t kBlocks = int64_t(1) << 22;  // of a launch: fewer than 2^32 threads

template <int DT, int TS>
hipError_t launch_turn(TurnArgs a, int64_t rows, unsigned threads, size_t lds, hipStream_t st) {
    const int64_t v_blocks = DT ? a.v_tiles * a.kv.seqs * a.Hk * ((a.D + kDims - 1) / kDims) : 0;
    int64_t n = 0, v = 0;
    while (n < rows || v < v_blocks) {
        const int64_t take = rows - n < kBlocks / a.bpt ? rows - n : kBlocks / a.bpt;
        const int64_t room = kBlocks - take * a.bpt, vtake = v_blocks - v < room ? v_blocks - v : room;
        a.row0 = n;
        a.turn_blocks = take * a.bpt;
        a.v0 = v;
        hipLaunchKernelGGL((turn_kernel<DT, TS>), dim3((unsigned)(a.turn_blocks + vtake)), dim3(threads), lds, st, a);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
        n += take;
        v += vtake;
    }
    return hipSuccess;
}

}  // namespace

hipError_t launch_rope(const float *X, int64_t x_stride, int64_t N, int64_t H, int64_t D, const int32_t *pos,
                       const float *freqs, int64_t rot, bool half, double mscale, float *Y, int64_t y_stride,
                       hipStream_t st) {
    TurnArgs a{};
    a.q = X;
    a.q_out = Y;
    a.q_stride = x_stride;
    a.out_stride = y_stride;
    a.pos = pos;
    a.freqs = freqs;
    a.mscale = mscale;
    a.Hq = (int)H;
    a.D = (int)D;
    a.rot = (int)rot;
    a.half = half;
    const int uph = (int)(D / 8);
    a.hpb = 256 / uph < H ? 256 / uph : (int)H;
    a.bpt = (int)((H + a.hpb - 1) / a.hpb);
    return launch_turn<0, 16>(a, N, (unsigned)((a.hpb * uph + 63) / 64 * 64), (size_t)rot / 2 * 16, st);
}

hipError_t launch_rope_freqs(int64_t rot, double base, double factor, double context, double fast, double slow,
                             const float *factors, float *freqs, hipStream_t st) {
    hipLaunchKernelGGL(freqs_kernel, dim3(1), dim3(512), 0, st, (int)rot, base, factor, context, fast, slow, factors, freqs);
    return hipGetLastError();
}

hipError_t launch_kv_append(const qmm_kv_cache &cache, const qmm_kv_batch &batch, const float *K, int64_t k_stride,
                            const float *V, int64_t v_stride, const float *freqs, int64_t rot, bool half, double mscale,
                            const int32_t *pos, const float *k_norm, const float *q_norm, double eps, const float *Q,
                            int64_t q_stride, int64_t q_heads, float *q_out, hipStream_t st) {
    TurnArgs a{};
    a.q = Q;
    a.k = K;
    a.v = V;
    a.q_out = q_out;
    a.q_stride = q_stride;
    a.k_stride = k_stride;
    a.v_stride = v_stride;
    a.out_stride = q_heads * cache.dim;
    a.pos = freqs ? pos : nullptr;
    a.freqs = freqs;
    a.q_norm = Q ? q_norm : nullptr;
    a.k_norm = k_norm;
    a.mscale = mscale;
    a.eps = eps;
    a.Hq = Q ? (int)q_heads : 0;
    a.Hk = cache.heads;
    a.D = cache.dim;
    a.rot = freqs ? (int)rot : 0;
    a.half = half;
    a.kv = kv_args(cache, batch);
    a.hpb = 256 / (a.D / 8);
    a.bpt = (a.Hq + a.Hk + a.hpb - 1) / a.hpb;
    const size_t turn_lds = (size_t)a.rot / 2 * 16 + 256 * 8 + (cache.dtype == QMM_Q8_0 ? 256 * 8 * 4 : 0);
    auto lds = [&](int ts) {
        const size_t tile = ((size_t)ts * kPitch + (size_t)ts * (kDims / 32)) * 4;
        return tile > turn_lds ? tile : turn_lds;
    };
    // tiles of 64 places (a 128-byte line of f16 places) for many new tokens, else of 16, which are more
    // workgroups: 8 x 512 tokens of 32/8 heads of 128 42.6 us (44.2 with 16), 8 x 64 9.4 (9.9 with 64),
    // 512 9.4 (9.8)
    const int ts = batch.seqs * batch.max_new < tuning_lever("QMM_APPEND_TILE_FROM", 2048) ? 16 : 64;
    a.v_tiles = (batch.max_new + 2 * ts - 2) / ts;
    const int64_t rows = batch.rows;
#define QMM_TURN(DT) \
    (ts == 16 ? launch_turn<DT, 16>(a, rows, 256, lds(16), st) : launch_turn<DT, 64>(a, rows, 256, lds(64), st))
    return cache.dtype == QMM_F16 ? QMM_TURN(QMM_F16) : QMM_TURN(QMM_Q8_0);
#undef QMM_TURN
}

}  // namespace qmm
