// tp_paged_index.h -- the index arithmetic of a paged key/value cache
// (tp_kv_cache): which rows of the projection buffer are a sequence's new
// tokens, where their positions live, the bounds checks of both, and the
// division of attention's work.  Plain C++, so that the host's tests run the
// code that the kernels run.
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

// ------------------------------------------------------------ attention's work
//
// A tile is R query rows of one sequence and KV head g: row r of the sequence's
// n * G (G query heads per KV head) is token r / G and query head g G + r % G,
// so that the heads that read the same keys share a tile.  Its work is the
// blocks of KB keys up to the last key that its last row sees, one at least (a
// tile that sees nothing still writes its zeros).  All tiles' blocks in the
// order (sequence, g, tile) are numbered 0 .. total - 1, and CTA c of a grid
// takes `per` of them from c * per on: equal shares whatever the lengths, and
// a long sequence spreads over the CTAs.  A tile cut by a share's border is
// written as partial results: by the CTA where it begins in that CTA's slot 1,
// by those that continue it in their slot 0.

struct Tiling {
    int rows, keys;  // R, KB
    int group;       // G
};

// Keys of sequence q that exist: its length, at most what the page table holds.
TP_HD int paged_keys(const PagedView& v, const PagedSeq& q) {
    const long long cap = static_cast<long long>(v.max_pages) << v.page_log2;
    return static_cast<int>(pmin(q.len, cap));
}

// Keys that row r of the sequence sees (none or fewer than none: nothing).
TP_HD int row_keys(const PagedSeq& q, int keys, long long r, int group) {
    const long long seen = q.len - q.n + r / group + 1;
    return static_cast<int>(seen < keys ? seen : keys);
}

TP_HD int seq_tiles(const PagedSeq& q, const Tiling& t) {
    return static_cast<int>((static_cast<long long>(q.n) * t.group + t.rows - 1) / t.rows);
}

TP_HD int tile_blocks(const PagedSeq& q, int keys, const Tiling& t, int tile) {
    const long long last = pmin((tile + 1ll) * t.rows, static_cast<long long>(q.n) * t.group) - 1;
    const int seen = row_keys(q, keys, last, t.group);
    return seen <= 0 ? 1 : (seen - 1) / t.keys + 1;
}

// Blocks of one KV head of a sequence.
TP_HD long long seq_blocks(const PagedView& v, const PagedSeq& q, const Tiling& t) {
    const int keys = paged_keys(v, q), nt = seq_tiles(q, t);
    long long sum = 0;
    for (int i = 0; i < nt; ++i) sum += tile_blocks(q, keys, t, i);
    return sum;
}

// A CTA's walk over its share: segments of consecutive blocks of one tile.
struct TileWalk {
    PagedSeq q;
    long long left;  // blocks of the share not yet taken
    int s, g, tile, tiles, keys;
    int kb, nkb;     // next block of the tile, its number of blocks

    // Begin `count` blocks at block `off` of sequence s0 (all KV heads counted).
    TP_HD void start(const PagedView& v, const Tiling& t, int s0, long long off, long long count) {
        left = count;
        s = s0;
        if (left <= 0) return;
        q = paged_seq(v, s);
        keys = paged_keys(v, q);
        tiles = seq_tiles(q, t);
        const long long per_head = seq_blocks(v, q, t);
        g = static_cast<int>(off / per_head);
        off -= g * per_head;
        tile = 0;
        nkb = tile_blocks(q, keys, t, 0);
        while (off >= nkb) {
            off -= nkb;
            ++tile;
            nkb = tile_blocks(q, keys, t, tile);
        }
        kb = static_cast<int>(off);
    }
    // Blocks of the current segment.
    TP_HD int segment() const { return static_cast<int>(pmin(left, nkb - kb)); }
    // Move past the current segment.
    TP_HD void next(const PagedView& v, const Tiling& t) {
        const int n = segment();
        left -= n;
        kb += n;
        if (left <= 0 || kb < nkb) return;
        kb = 0;
        if (++tile == tiles) {
            tile = 0;
            if (++g == v.kv_heads) {
                g = 0;
                do {
                    if (++s >= v.n_seqs) {  // cannot be: the share ends inside the work
                        left = 0;
                        return;
                    }
                    q = paged_seq(v, s);
                } while (q.n == 0);
                keys = paged_keys(v, q);
                tiles = seq_tiles(q, t);
            }
        }
        nkb = tile_blocks(q, keys, t, tile);
    }
};

}  // namespace tpk
