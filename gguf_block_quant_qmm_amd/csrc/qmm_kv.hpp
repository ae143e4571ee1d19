// qmm_kv.hpp -- the paged key-value cache (include/qmm.h, qmm_kv_cache and
// qmm_kv_batch) as the kernels see it.  Included only by the HIP sources.
#pragma once

#include "qmm_device.hpp"

namespace qmm {

struct KvArgs {
    uint8_t *k, *v;
    const int32_t *table, *lens, *starts;
    int64_t table_stride;
    int pages, max_pages, heads, page_shift, seqs, max_new, rows;
};

inline KvArgs kv_args(const qmm_kv_cache &c, const qmm_kv_batch &b) {
    KvArgs a;
    a.k = (uint8_t *)c.k;
    a.v = (uint8_t *)c.v;
    a.table = b.table;
    a.lens = b.lens;
    a.starts = b.starts;
    a.table_stride = b.table_stride ? b.table_stride : b.max_pages;
    a.pages = (int)c.pages;
    a.max_pages = (int)b.max_pages;
    a.heads = c.heads;
    a.page_shift = __builtin_ctz((unsigned)c.page);
    a.seqs = (int)b.seqs;
    a.max_new = (int)b.max_new;
    a.rows = (int)b.rows;
    return a;
}

// Bytes of the record of one page of one head in either pool.
__host__ __device__ inline int64_t kv_record(int dtype, int64_t page, int64_t dim) {
    return dtype == QMM_F16 ? 2 * page * dim : page * dim + page * dim / 16;
}

// The new tokens of sequence s: rows first .. first + count - 1 of the call's
// arrays, token t of them at index `index + t` of the sequence.  count is cut to
// what the arrays hold and to max_new; the index is not moved by that.
struct KvNew {
    int first, count;
    int64_t index, len;
};
__host__ __device__ __forceinline__ KvNew kv_new(const KvArgs &a, int s) {
    KvNew r;
    r.len = a.lens[s];
    int64_t first, n;
    if (a.starts) {
        first = a.starts[s];
        n = (int64_t)a.starts[s + 1] - first;
    } else {
        first = (int64_t)s * a.max_new;
        n = a.max_new;
    }
    r.index = r.len - n;
    if (first < 0) n = 0;
    n = n < a.max_new ? n : a.max_new;
    n = n < a.rows - first ? n : a.rows - first;
    r.first = (int)first;
    r.count = n > 0 ? (int)n : 0;
    return r;
}

// The sequence of row n (uniform over the wavefront), or -1 for padding.  With
// starts, sequence s ends before starts[s + 1]: the count of ends at or below n,
// 64 at a time, all loads of a round at once.
__device__ __forceinline__ int kv_row_seq(const KvArgs &a, int n) {
    int s;
    if (a.starts) {
        if (n < a.starts[0]) return -1;
        s = 0;
        const int lane = (int)threadIdx.x & 63;
        for (int b = 0; b < a.seqs; b += 64) {
            const bool below = b + lane < a.seqs && a.starts[b + lane + 1] <= n;
            const int got = __popcll(__ballot(below));
            s += got;
            if (got < 64) break;
        }
    } else {
        s = n / a.max_new;
    }
    return s < a.seqs ? __builtin_amdgcn_readfirstlane(s) : -1;
}

// The page of token i (i >= 0) of sequence s, or -1 if it has none.
__host__ __device__ __forceinline__ int kv_page(const KvArgs &a, int s, int64_t i) {
    const int64_t c = i >> a.page_shift;
    if (i < 0 || c >= a.max_pages) return -1;
    const int p = a.table[(int64_t)s * a.table_stride + c];
    return p >= 0 && p < a.pages ? p : -1;
}

}  // namespace qmm
