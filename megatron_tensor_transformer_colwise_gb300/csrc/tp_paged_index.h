// tp_paged_index.h -- the index arithmetic of a paged key/value cache
// (tp_kv_cache): which rows of the projection buffer are a sequence's new
// tokens, where their positions live, the bounds checks of both, and the
// division of attention's work.  Plain C++, so that the host's tests run the
// code that the kernels run.
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define TP_HD __host__ __device__ __forceinline__
// Run once a tile or less, and kept out of line: inlined into every role of a
// kernel they outgrew the instruction cache.
#define TP_HD_CALL __host__ __device__ __noinline__ inline
#else
#define TP_HD inline
#define TP_HD_CALL inline
#endif

namespace tpk {

TP_HD long long pmin(long long a, long long b) { return a < b ? a : b; }
TP_HD long long pmax(long long a, long long b) { return a > b ? a : b; }

TP_HD int imin(int a, int b) { return a < b ? a : b; }
TP_HD int imax(int a, int b) { return a > b ? a : b; }

// Longest sequence: positions and their block ends stay in 32 bits.
constexpr int kMaxLen = 1 << 30;

struct PagedView {
    const int32_t* table;    // [n_seqs][max_pages]
    const int32_t* q_start;  // [n_seqs + 1]
    const int32_t* kv_len;   // [n_seqs]
    long long n_pages;
    int rows;                // M
    int n_seqs, max_pages, page_log2;
    int kv_heads, d;
};

// A sequence's rows and lengths, clamped to what exists: the i-th of its n new
// tokens is row row0 + i, at position len - n + i (negative: sees nothing).
struct PagedSeq {
    int row0, n, len;
};

TP_HD PagedSeq paged_seq(const PagedView& v, int s) {
    const int a = imin(imax(v.q_start[s], 0), v.rows), b = imin(imax(v.q_start[s + 1], a), v.rows);
    PagedSeq x;
    x.row0 = a;
    x.n = b - a;
    x.len = imin(imax(v.kv_len[s], 0), kMaxLen);
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
TP_HD int paged_owner(const int32_t* q_start, int n_seqs, int row) {
    if (n_seqs == 0 || row < q_start[0] || row >= q_start[n_seqs]) return -1;
    int lo = 0, hi = n_seqs;  // q_start[lo] <= row < q_start[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (q_start[mid] <= row) lo = mid;
        else hi = mid;
    }
    return lo;
}

// ------------------------------------------------------------ attention's work
//
// A tile is `tok` new tokens of one sequence with the G = a/k query heads of
// one KV head g: row r is token r / G and query head g G + r % G, so that the
// heads that read the same keys share a tile.  Its work is the blocks of KB
// keys up to the last key that its last token sees, one at least (a tile that
// sees nothing still writes its zeros).  All tiles' blocks in the order
// (sequence, g, tile) are numbered 0 .. total - 1, and CTA c of a grid takes
// `per` of them from c * per on: equal shares whatever the lengths, and a long
// sequence spreads over the CTAs.  A tile cut by a share's border is written as
// partial results: by the CTA where it begins in that CTA's slot 1, by those
// that continue it in their slot 0.

struct Tiling {
    int tok, group;  // tokens of a tile, G
    int log2_keys;   // KB = 2^log2_keys
    int log2_tok;    // log2 of tok, -1 if that is not a power of two (at most KB)
    int least = 1, most = 0x7fffffff;  // new tokens of the sequences that are taken; the others are as if they had none
};

inline int exact_log2(int x) {
    int k = 0;
    while ((1 << k) < x) ++k;
    return (1 << k) == x ? k : -1;
}

// Keys of sequence q that exist: its length, at most what the page table holds.
TP_HD int paged_keys(const PagedView& v, const PagedSeq& q) {
    return static_cast<int>(pmin(q.len, static_cast<long long>(v.max_pages) << v.page_log2));
}

// Keys that token i of the sequence sees (none or fewer than none: nothing).
TP_HD int token_keys(const PagedSeq& q, int keys, int i) {
    const int seen = q.len - q.n + i + 1;
    return seen < keys ? seen : keys;
}

TP_HD bool taken(const PagedSeq& q, const Tiling& t) { return q.n >= t.least && q.n <= t.most; }

TP_HD unsigned by_tok(unsigned x, const Tiling& t) { return t.log2_tok >= 0 ? x >> t.log2_tok : x / static_cast<unsigned>(t.tok); }
TP_HD int seq_tiles(const PagedSeq& q, const Tiling& t) { return static_cast<int>(by_tok(static_cast<unsigned>(q.n + t.tok - 1), t)); }

// Tokens of a tile that are the sequence's.
TP_HD int tile_tokens(const PagedSeq& q, const Tiling& t, int tile) {
    const int left = q.n - tile * t.tok;
    return left < t.tok ? left : t.tok;
}

TP_HD int tile_blocks(const PagedSeq& q, int keys, const Tiling& t, int tile) {
    const int seen = token_keys(q, keys, tile * t.tok + tile_tokens(q, t, tile) - 1);
    return seen <= 0 ? 1 : ((seen - 1) >> t.log2_keys) + 1;
}

// sum_{x < n} floor(x / 2^k).
TP_HD long long quotient_sum(unsigned n, int k) {
    const unsigned q = n >> k, r = n & ((1u << k) - 1);
    if (n < 65536u) return static_cast<long long>(((q * (q - 1) / 2) << k) + r * q);  // below n^2
    return ((static_cast<long long>(q) * (q - 1) / 2) << k) + static_cast<long long>(r) * q;
}

// sum_{x < n} floor((a x + b) / m), by Euclid's algorithm on (m, a).  a n + b
// stays below 2^32 here: it starts at the sequence's tokens and a block of
// keys, and never grows.
TP_HD long long floor_sum(unsigned n, unsigned m, unsigned a, unsigned b) {
    long long sum = 0;
    while (n > 0) {
        sum += static_cast<long long>(n) * (n - 1) / 2 * (a / m) + static_cast<long long>(n) * (b / m);
        a %= m;
        const unsigned top = a * n + b % m;
        n = top / m;
        b = top % m;
        const unsigned x = m;
        m = a;
        a = x;
        if (m == 0) break;
    }
    return sum;
}

// Blocks of the first `count` tiles of one KV head of a sequence.
TP_HD_CALL long long tiles_blocks(const PagedSeq q, int keys, const Tiling t, int count) {
    if (count <= 0) return 0;
    long long sum = 0;
    if (count == seq_tiles(q, t)) sum += tile_blocks(q, keys, t, --count);  // the last tile may be short
    // Tile j sees up to e_j = base + (j + 1) tok: one block while e_j <= KB, ceil(e_j / KB) while e_j < keys,
    // then ceil(keys / KB).
    const int base = q.len - q.n, kb = 1 << t.log2_keys;
    const unsigned tok = static_cast<unsigned>(t.tok);
    const unsigned one = kb < base ? 0u : by_tok(static_cast<unsigned>(kb - base), t);
    const unsigned full = keys <= base ? 0u : by_tok(static_cast<unsigned>(keys) - static_cast<unsigned>(base) - 1u, t);
    const unsigned n = static_cast<unsigned>(count);
    const unsigned c1 = one < n ? one : n;
    const unsigned c2 = full < c1 ? c1 : full < n ? full : n;
    sum += c1;
    if (c2 > c1) {
        const unsigned b = static_cast<unsigned>(base + kb - 1) + (c1 + 1) * tok;
        if (t.log2_tok >= 0) {  // floor((tok x + b) / KB) = floor((x + floor(b / tok)) / (KB / tok))
            const unsigned y = b >> t.log2_tok;
            sum += quotient_sum(c2 - c1 + y, t.log2_keys - t.log2_tok) - quotient_sum(y, t.log2_keys - t.log2_tok);
        } else {
            sum += floor_sum(c2 - c1, 1u << t.log2_keys, tok, b);
        }
    }
    const int most = keys <= 0 ? 1 : ((keys - 1) >> t.log2_keys) + 1;
    return sum + static_cast<long long>(n - c2) * most;
}

// Blocks of a sequence, one KV head.
TP_HD long long head_blocks(const PagedView& v, const PagedSeq& q, const Tiling& t) {
    if (!taken(q, t)) return 0;
    const int keys = paged_keys(v, q);
    return q.n <= t.tok ? tile_blocks(q, keys, t, 0) : tiles_blocks(q, keys, t, seq_tiles(q, t));
}

// Blocks of a sequence, all KV heads.
TP_HD long long seq_blocks(const PagedView& v, const PagedSeq& q, const Tiling& t) {
    return head_blocks(v, q, t) * static_cast<long long>(v.kv_heads);
}

// A CTA's walk over its share: segments of consecutive blocks of one tile.
struct TileWalk {
    PagedSeq q;
    long long left;  // blocks of the share not yet taken
    int s, g, tile, tiles, keys;
    int kb, nkb;     // next block of the tile, its number of blocks

    // Blocks of the current segment.
    TP_HD int segment() const { return static_cast<int>(pmin(left, nkb - kb)); }
    // Move past the current segment.
    TP_HD_CALL void next(const PagedView& v, const Tiling& t) {
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
                } while (!taken(q, t));
                keys = paged_keys(v, q);
                tiles = seq_tiles(q, t);
            }
        }
        nkb = tile_blocks(q, keys, t, tile);
    }
};

}  // namespace tpk
