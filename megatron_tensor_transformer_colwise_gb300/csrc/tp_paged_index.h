// tp_paged_index.h -- the index arithmetic of a paged key/value cache
// (tp_kv_cache): which rows of the projection buffer are a sequence's new
// tokens, where their positions live, and the bounds checks of both.  Plain
// C++, so that the host's tests run the code that the kernels run.
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define TP_HD __host__ __device__ __forceinline__
#else
#define TP_HD inline
#endif

namespace tpk {

TP_HD long long pmin(long long a, long long b) { return a < b ? a : b; }
TP_HD long long pmax(long long a, long long b) { return a > b ? a : b; }

// Longest sequence: positions and their block ends stay in 32 bits.
constexpr int kMaxLen = 1 << 30;

struct PagedView {
    const int32_t* table;    // [n_seqs][max_pages]
    const int32_t* q_start;  // [n_seqs + 1]
    const int32_t* kv_len;   // [n_seqs]
    long long n_pages;
    long long rows;          // M
    int n_seqs, max_pages, page_log2;
    int kv_heads, d;
};

// A sequence's rows and lengths, clamped to what exists: the i-th of its n new
// tokens is row row0 + i, at position len - n + i (negative: sees nothing).
struct PagedSeq {
    long long row0;
    int n;
    int len;
};

TP_HD PagedSeq paged_seq(const PagedView& v, int s) {
    const long long a = pmin(pmax(v.q_start[s], 0), v.rows);
    const long long b = pmin(pmax(v.q_start[s + 1], a), v.rows);
    PagedSeq x;
    x.row0 = a;
    x.n = static_cast<int>(b - a);
    x.len = static_cast<int>(pmin(pmax(v.kv_len[s], 0), kMaxLen));
    return x;
}

// Page of position pos of sequence s, or -1 where it is not in the cache.
TP_HD long long paged_page(const PagedView& v, int s, int pos) {
    const int i = pos >> v.page_log2;
    if (pos < 0 || i >= v.max_pages) return -1;
    const long long pg = v.table[static_cast<long long>(s) * v.max_pages + i];
    return (pg >= 0 && pg < v.n_pages) ? pg : -1;
}

// Index of the (page, KV head, offset) row of the cache, in rows of d elements
// (and in scales).  64 bits: a cache passes 2^31 elements.
TP_HD long long paged_row(const PagedView& v, long long page, int g, int pos) {
    return ((page * v.kv_heads + g) << v.page_log2) + (pos & ((1 << v.page_log2) - 1));
}

// Sequence that owns `row`: the last s with q_start[s] <= row, if the row is
// below q_start[s + 1]; -1 otherwise.
TP_HD int paged_owner(const PagedView& v, long long row) {
    int lo = 0, hi = v.n_seqs;  // invariant: q_start[lo] <= row (if any), q_start[hi] > row
    if (v.n_seqs == 0 || row < v.q_start[0] || row >= v.q_start[v.n_seqs]) return -1;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (v.q_start[mid] <= row) lo = mid;
        else hi = mid;
    }
    return lo;
}

}  // namespace tpk
