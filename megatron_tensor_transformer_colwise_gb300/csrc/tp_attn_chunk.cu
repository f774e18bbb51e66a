// tp_attn_chunk.cu -- causal GQA attention of new tokens over a paged
// key/value cache, many query rows per sequence and KV head: chunks of
// prompts, long drafts, and mixtures of those with single tokens.
//
// The mathematics is that of tp_attn_paged.cu (one pass over the keys with a
// running maximum and sum a row).  A tile is 128 query rows, the G = a/k heads
// of a KV head next to each other for each token, so that a key block read
// once serves all of them; 4 * 128 * d operations a key against 4 d bytes: the
// tensor cores bound it as soon as a tile is full.  The work is cut into equal
// shares of 128-key blocks (tp_paged_index.h), one persistent CTA an SM:
//   warp 0      TMA: Q of a tile as one box {64, heads, shards, tokens}, K blocks
//               as one box a page and 64 columns.
//   warp 1      TMEM owner and S issuer: S = Q K^T (tcgen05, fp32) into three
//               TMEM buffers.
//   warp 2      PV issuer: O += P V, P from tensor memory.
//   warp 3      TMA: V blocks.  A copy takes its issuing thread about 150
//               cycles here (its operands go to uniform registers one by one),
//               so K and V have a thread each; page numbers are read 32 at a
//               time, a window ahead.
//   warps 4..11 softmax, two warps a TMEM lane quadrant, half of a block's keys
//               each; a tile's outputs leave after the next tile's first block.
// From an 8-bit cache the codes of K and V come through a ring of their own
// (warp 0 loads both), and warps 12..15 write them out as bf16, which holds
// every code, in the layout the products read.  The scales stay outside the
// products, as in tp_attn_paged.cu: K's multiplies S's columns, V's the columns
// of P before P is rounded to bf16.
//
// P is rounded to bf16 because a product's operands have one type and V is bf16:
// at most 2^-8 of each weight, at random, while sums, maxima and O stay in fp32.  The
// outputs are off by 0.0023 of their size where one rounding at the end gives
// 0.0017.  With V's scale in P, weights below 2^-126 / scale lose bits; a scale is
// 2^-109 at least as the cache writes them, so that such a weight is below 2^-17.
//
// Measured, 32 query heads on 8 KV heads of 128: 2048 tokens behind 8192 cached
// ones 249 us with fresh inputs (0.67 of cuBLAS's rate for the keys that are seen),
// 236 us, 1300 TFLOP/s and 0.70 with the same inputs again.  A block of
// 128 keys then takes 1900 cycles where its products need 1024: the softmax bounds
// it (eight warps: maximum, 2^x, rounding and the way through tensor memory).
// From 8 bits a block takes 1.7 us instead of 1.1: the converting warps share the
// schedulers and shared memory with the softmax.  fp16 instead of bf16 would take
// half the conversion's instructions, but Q has to become fp16 once a tile and P's
// range has to be watched (2.6 us a block as built, where bf16 took 2.1).  With 512
// threads the roles have 128 registers, and what spills costs more than arithmetic.
// A tile costs 1 to 3 us besides its blocks (Q, first page, last output) and a CTA's
// first about 3, which is what short contexts pay.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstring>
#include <string>

#include "tp_attn_paged.cuh"
#include "tp_packed.cuh"

namespace {

using namespace tpk;

constexpr int QB = 128;          // TMEM lanes: rows of a tile, at most
constexpr int KB = 128;          // keys of a block
constexpr int NS = 3;            // S buffers in TMEM
constexpr int BOX = 128 * 128;   // 128 rows of one swizzle span (64 bf16)
constexpr float RESCALE = 8.0f;  // log2 of the growth of P before O is rescaled

enum {
    B_Q_FULL = 0,
    B_Q_EMPTY = 1,
    B_K_FULL = 2,    // x2
    B_K_EMPTY = 4,   // x2
    B_V_FULL = 6,    // x2
    B_V_EMPTY = 8,   // x2
    B_S_FULL = 10,               // x NS
    B_PV_DONE = B_S_FULL + NS,   // x NS: the PV product that read P from buffer i has completed
    B_P_FULL = B_PV_DONE + NS,   // x NS
    B_O_FULL = B_P_FULL + NS,
    B_O_EMPTY = B_O_FULL + 1,
    B_DRAIN = B_O_EMPTY + 1,     // x2
    B_R_FULL = B_DRAIN + 2,      // x NRAW: codes of a K or V block
    B_R_EMPTY = B_R_FULL + 3,
    B_SC_FULL = B_R_EMPTY + 3,   // x NSC: scales of a block
    NUM_BARS = B_SC_FULL + 4
};
constexpr int NRAW = 3;  // stages of the ring of codes
constexpr int NSC = 4;   // blocks whose scales are held (a block's codes are loaded once PV of the fourth before it is done)

// What the epilogue of a segment needs once its walk has moved on.
struct Done {
    int row0, g, rows, where;  // row0: the tile's first token's row; where: -1 the output, else the CTA's slot
};

template <int D_, bool E4M3_>
struct Lay {
    static constexpr int D = D_;
    static constexpr bool E4M3 = E4M3_;
    static constexpr int NT = E4M3 ? 512 : 384;
    static constexpr int KRING = E4M3 ? NRAW : 2;   // stages that the producers fill
    static constexpr int FULL = E4M3 ? 4 : 1;       // arrivals that fill an operand stage: converting warps, or the copy
    static constexpr int CODES = KB * D;            // bytes of a block's codes
    static constexpr int RAW = E4M3 ? CODES + 2 * KB * 4 : 0;  // and, behind K's, the block's scales of K and V
    static constexpr int NSEG = D / 64;
    static constexpr int TILE = KB * D * 2;  // Q, K or V
    static constexpr int Q_OFF = 0;
    static constexpr int K_OFF = TILE;
    static constexpr int V_OFF = K_OFF + 2 * TILE;
    static constexpr int DC = D / 2;         // O columns of a softmax warp
    static constexpr int STG_ROW = DC * 2;            // bytes of a staged output row
    static constexpr int STG_OFF = V_OFF + 2 * TILE;  // 32 rows a softmax warp
    static constexpr int RAW_OFF = STG_OFF + (E4M3 ? 0 : 8 * 32 * STG_ROW);  // no room for staged outputs beside the codes
    static constexpr int SC_OFF = RAW_OFF + NRAW * RAW;
    static constexpr int XCH_OFF = SC_OFF + (E4M3 ? NSC * 2 * KB * 4 : 0);  // [9][128] fp32: maxima and sums, each by parity and half; references
    static constexpr int BAR_OFF = XCH_OFF + 9 * QB * 4;
    static constexpr int SCAN_OFF = BAR_OFF + 8 * NUM_BARS + 16;
    static constexpr int WALK_OFF = SCAN_OFF + 8 * (NT / 32 + 2);  // one walk a warp, and the producers' ahead
    static constexpr int DONE_OFF = WALK_OFF + (NT / 32 + 2) * sizeof(TileWalk);
    static constexpr int PAGE_OFF = (DONE_OFF + 8 * sizeof(Done) + 15) / 16 * 16;  // page numbers of the two producers
    static constexpr int DATA = PAGE_OFF + 2 * 64 * 4;
    static constexpr int SMEM = DATA + 1024;
    static constexpr int O_COL = NS * KB;
    static constexpr int P_HALF = E4M3 ? KB / 2 : KB / 4;  // columns between P's halves of a block's keys
    static_assert(O_COL + D <= 512 && SMEM <= 232448 && SCAN_OFF % 8 == 0 && sizeof(TileWalk) % 8 == 0, "configuration");
};

struct Params {
    const float *k_scale, *v_scale;
    CUtensorMap map_q;         // the projection buffer as {d, heads a shard, shards, tokens}
    CUtensorMap map_k, map_v;  // the cache as {d, page, k, n_pages}
    CUtensorMap map_o;         // O as {d, heads, tokens}, boxes of 32 rows of a KV head and half their columns
    int o_boxes;               // 1: G divides 32, so that such a box is whole tokens
    PagedView v;
    __nv_bfloat16* o;
    int heads, group, tile_tok, log2_tok, box_rows, least, most;
    int kv_per_shard;        // KV heads of a shard, 0 if shards share them
    int shards_per_kv;       // shards that share a KV head (1 if they have their own)
    float scale_log2;
    float* part_o;   // [grid][2] slots of 128 rows in 16-byte pieces, as the join reads them
    float* part_ml;
    int4* desc;
    unsigned* status;
    unsigned long long timeout_ns;
};

template <class L>
__global__ void __launch_bounds__(L::NT, 1) attn_chunk_kernel(const __grid_constant__ Params p) {
    constexpr int D = L::D, NSEG = L::NSEG, NT = L::NT;
    constexpr bool E4M3 = L::E4M3;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t* gbase = smem_raw + (base - raw);
    const uint32_t sQ = base + L::Q_OFF, sK = base + L::K_OFF, sV = base + L::V_OFF;
    auto bar = [&](int i) { return base + L::BAR_OFF + 8u * static_cast<uint32_t>(i); };
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(gbase + L::BAR_OFF + 8 * NUM_BARS);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const Tiling tiling = {p.tile_tok, p.group, 7, p.log2_tok, p.least, p.most};
    const Waiter wait = {abort_flag, p.status, p.timeout_ns};

    if (threadIdx.x == 0) {
        mbar_init(bar(B_Q_FULL), 1);
        mbar_init(bar(B_Q_EMPTY), 1);
        for (int s = 0; s < 2; ++s) {
            mbar_init(bar(B_K_FULL + s), L::FULL);
            mbar_init(bar(B_K_EMPTY + s), 1);
            mbar_init(bar(B_V_FULL + s), L::FULL);
            mbar_init(bar(B_V_EMPTY + s), 1);
        }
        for (int s = 0; s < NS; ++s) {
            mbar_init(bar(B_S_FULL + s), 1);
            mbar_init(bar(B_PV_DONE + s), 1);
            mbar_init(bar(B_P_FULL + s), 8);
        }
        mbar_init(bar(B_O_FULL), 1);
        mbar_init(bar(B_O_EMPTY), 8);
        mbar_init(bar(B_DRAIN), 1);
        mbar_init(bar(B_DRAIN + 1), 1);
        for (int s = 0; s < NRAW; ++s) {
            mbar_init(bar(B_R_FULL + s), 1 + 32);  // the codes' copies, and the lanes that copy scales
            mbar_init(bar(B_R_EMPTY + s), 4);
        }
        for (int s = 0; s < NSC; ++s) mbar_init(bar(B_SC_FULL + s), 4);
        *abort_flag = 0;
        fence_barrier_init();
        tma_prefetch_desc(&p.map_q);
        tma_prefetch_desc(&p.map_k);
        tma_prefetch_desc(&p.map_v);
    }
    if (warp == 1) {
        tmem_alloc(smem_u32(tmem_slot), 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    pdl_trigger();
    pdl_wait();
    TileWalk* walks = reinterpret_cast<TileWalk*>(gbase + L::WALK_OFF);
    TileWalk& w = walks[warp];  // each warp walks on its own, in shared memory; lane 0 moves
    const Share share = find_share<L::NT>(p.v, tiling, reinterpret_cast<long long*>(gbase + L::SCAN_OFF), w);
    const uint32_t tmem = *tmem_slot;
    auto move_on = [&] {
        __syncwarp();
        if (lane == 0) w.next(p.v, tiling);
        __syncwarp();
    };

    if (warp == 0 || (warp == 3 && !E4M3)) {
        // ---------------------------------------------------------- TMA producers
        const bool is_v = warp == 3;
        const int log2 = p.v.page_log2, per_block = KB / p.box_rows;
        // Page numbers of two windows of 32 pages: page i of the sequence at ring[i - first page of the segment, mod 64].
        int* ring = reinterpret_cast<int*>(gbase + L::PAGE_OFF) + (is_v ? 64 : 0);
        const uint32_t dst0 = E4M3 ? base + L::RAW_OFF : is_v ? sV : sK;
        const uint32_t full0 = bar(E4M3 ? B_R_FULL : is_v ? B_V_FULL : B_K_FULL);
        const uint32_t empty0 = bar(E4M3 ? B_R_EMPTY : is_v ? B_V_EMPTY : B_K_EMPTY);
        int4 cut = make_int4(0, 0, 0, 0);  // the tile that begins here and goes on in the next CTAs
        uint32_t n = 0, li = 0;            // blocks and Q tiles issued
        bool ok = true;
        // Page i of a segment's sequence; -1: past its keys, or on no page of the cache.
        auto page_at = [&](const TileWalk& x, int i) -> int {
            if ((static_cast<long long>(i) << log2) >= x.keys) return -1;
            const int pg = p.v.table[static_cast<long long>(x.s) * p.v.max_pages + i];
            if (pg >= 0 && pg < p.v.n_pages) return pg;
            if (p.status) atomicOr(p.status, kStatusPage);
            return -1;
        };
        // y walks a segment ahead: the first pages of the next segment are read, and its Q is brought to L2, in time.
        TileWalk& y = walks[NT / 32 + (is_v ? 1 : 0)];
        if (lane == 0) y = w;
        __syncwarp();
        auto q_box = [&](const TileWalk& x, bool load) {
            const int head = p.kv_per_shard ? (x.g % p.kv_per_shard) * p.group : 0;
            const int shard = p.kv_per_shard ? x.g / p.kv_per_shard : x.g * p.shards_per_kv;
            const int token = x.q.row0 + x.tile * p.tile_tok;
#pragma unroll 1
            for (int c = 0; c < NSEG; ++c) {
                if (load) tma_load_4d(sQ + c * BOX, &p.map_q, bar(B_Q_FULL), 64 * c, head, shard, token);
                else tma_prefetch_l2_4d(&p.map_q, 64 * c, head, shard, token);
            }
        };
        int first = -1, behind = -1;
        if (y.left > 0) {
            first = page_at(y, ((y.kb * KB) >> log2) + lane);
            behind = page_at(y, ((y.kb * KB) >> log2) + 32 + lane);
        }
        while (y.left > 0 && ok) {
            __syncwarp();
            if (lane == 0) {
                w = y;
                y.next(p.v, tiling);
            }
            __syncwarp();
            const int seg = w.segment(), g = w.g, page0 = (w.kb * KB) >> log2;
            int next = behind;
            ring[lane] = first;
            __syncwarp();
            if (y.left > 0) {
                first = page_at(y, ((y.kb * KB) >> log2) + lane);
                behind = page_at(y, ((y.kb * KB) >> log2) + 32 + lane);
                if (!is_v && lane == 0) q_box(y, false);
            }
            if (w.kb == 0 && seg < w.nkb) {
                const long long at = share.begin + share.count - seg;  // the segment is the share's last
                cut = make_int4(w.q.row0 + w.tile * p.tile_tok, g, tile_tokens(w.q, tiling, w.tile) * p.group,
                                share_of(at + w.nkb - 1, share.per) - static_cast<int>(blockIdx.x) + 1);
            }
            for (int i = 0, at = 0; i < seg && ok; ++i, at += per_block) {
                if ((at & 31) == 0) {  // a window begins: the one behind it takes the other half of the ring
                    ring[(at + 32 + lane) & 63] = next;
                    if (i + 32 / per_block < seg) next = page_at(w, page0 + at + 64 + lane);
                    __syncwarp();
                }
#pragma unroll 1
                for (int kind = 0; kind < (E4M3 ? 2 : 1); ++kind, ++n) {  // 8 bits: K, then V
                    const uint32_t st = n % L::KRING;
                    ok = __all_sync(0xffffffffu, wait(empty0 + 8 * st, ((n / L::KRING) & 1u) ^ 1u));
                    if (!ok) break;
                    const uint32_t full = full0 + 8 * st;
                    if constexpr (E4M3) {
                        const uint32_t dst = dst0 + st * L::RAW;
                        // The block's scales of K and V behind K's codes, four keys a lane (of one page: it has 16 keys at
                        // least); those of no page are zeros.  With two copies a page by the issuing thread 3 chunks of
                        // 500 tokens over 8000 keys took 526 us at 16 keys a page and 369 at 32, so 366 and 303.
                        const int key = lane * 4, page = ring[(at + (key >> log2)) & 63];
                        const uint32_t sc = dst + L::CODES + key * 4;
                        if (kind == 0 && page >= 0) {
                            const long long row = paged_row(p.v, page, g, key & ((1 << log2) - 1));
                            copy16(sc, p.k_scale + row);
                            copy16(sc + KB * 4, p.v_scale + row);
                            copies_arrive(full);
                        } else {
                            if (kind == 0) {
                                st_shared_v4(sc, 0, 0, 0, 0);
                                st_shared_v4(sc + KB * 4, 0, 0, 0, 0);
                            }
                            mbar_arrive(full);
                        }
                        if (lane == 0) {
                            const CUtensorMap* map = kind ? &p.map_v : &p.map_k;
                            mbar_arrive_expect_tx(full, L::CODES);
#pragma unroll 1
                            for (int b = 0; b < per_block; ++b) {
                                const int page = ring[(at + b) & 63];
                                tma_load_4d(dst + b * p.box_rows * D, map, full, 0, 0, g, page);
                            }
                        }
                    } else if (lane == 0) {
                        const uint32_t dst = dst0 + st * L::TILE;
                        const CUtensorMap* map = is_v ? &p.map_v : &p.map_k;
                        mbar_arrive_expect_tx(full, L::TILE);
#pragma unroll 2
                        for (int b = 0; b < per_block; ++b) {
                            const int page = ring[(at + b) & 63];  // -1: TMA fills the box with zeros and reads nothing
#pragma unroll
                            for (int c = 0; c < NSEG; ++c)
                                tma_load_4d(dst + c * BOX + b * p.box_rows * 128, map, full, c * 64, 0, g, page);
                        }
                    }
                    __syncwarp();
                    if (!is_v && i == 0 && kind == 0) {  // Q behind the first K: it waits for the previous segment's last S
                        ok = __all_sync(0xffffffffu, li == 0 || wait(bar(B_Q_EMPTY), (li - 1) & 1u));
                        if (!ok) {
                            ++n;
                            break;
                        }
                        if (lane == 0) {
                            mbar_arrive_expect_tx(bar(B_Q_FULL), p.tile_tok * p.group * D * 2);
                            q_box(w, true);
                        }
                        ++li;
                        __syncwarp();
                    }
                }
            }
        }
        if (!is_v && lane == 0) p.desc[blockIdx.x] = cut;
        // No copy may be in flight when the CTA's shared memory goes.
        if constexpr (E4M3) copies_wait();
        if (!is_v && li) drain(bar(B_Q_FULL), (li - 1) & 1u);
        for (uint32_t i = n > L::KRING ? n - L::KRING : 0; i < n; ++i) drain(full0 + 8 * (i % L::KRING), (i / L::KRING) & 1u);
    } else if (warp == 1) {
        // ---------------------------------------------------------- S issuer
        if (lane == 0) {
            constexpr uint32_t idesc = idesc_bf16_f32(QB, KB);
            const uint64_t qdesc = sdesc_sw128(sQ), kdesc0 = sdesc_sw128(sK);
            bool ok = true;
            uint32_t gb = 0, li = 0;
            for (; w.left > 0 && ok; w.next(p.v, tiling), ++li) {
                const int seg = w.segment();
                ok = wait(bar(B_Q_FULL), li & 1u);
                for (int i = 0; i < seg && ok; ++i, ++gb) {
                    const uint32_t st = gb & 1u, sb = gb % NS;
                    // Buffer sb held P of block gb - NS: its PV must have read it.
                    ok = (gb < NS || wait(bar(B_PV_DONE + sb), ((gb - NS) / NS) & 1u)) &&
                         wait(bar(B_K_FULL + st), (gb >> 1) & 1u);
                    if (!ok) break;
                    tc_fence_after();
                    const uint64_t kdesc = kdesc0 + (st * L::TILE) / 16;
#pragma unroll
                    for (int ks = 0; ks < D / 16; ++ks) {
                        const uint32_t off = ((ks >> 2) * BOX + (ks & 3) * 32) / 16;
                        umma_bf16(tmem + sb * KB, qdesc + off, kdesc + off, idesc, ks > 0 ? 1u : 0u);
                    }
                    umma_commit(bar(B_K_EMPTY + st));
                    umma_commit(bar(B_S_FULL + sb));
                }
                if (ok) umma_commit(bar(B_Q_EMPTY));
            }
            // Every product has completed before TMEM and shared memory go.
            umma_commit(bar(B_DRAIN));
            drain(bar(B_DRAIN), 0);
        }
    } else if (warp == 2) {
        // ---------------------------------------------------------- PV issuer
        if (lane == 0) {
            constexpr uint32_t idesc = idesc_bf16_f32_bmn(QB, D);
            const uint64_t vdesc0 = sdesc_sw128_mn(sV, BOX, 1024);
            bool ok = true;
            uint32_t gb = 0, li = 0;
            for (; w.left > 0 && ok; w.next(p.v, tiling), ++li) {
                const int seg = w.segment();
                for (int i = 0; i < seg && ok; ++i, ++gb) {
                    const uint32_t st = gb & 1u, pb = gb % NS;
                    ok = wait(bar(B_P_FULL + pb), (gb / NS) & 1u) &&
                         wait(bar(B_V_FULL + st), (gb >> 1) & 1u);
                    // The first PV of a segment overwrites O: the previous epilogue must have read it.
                    if (ok && i == 0 && li > 0)
                        ok = wait(bar(B_O_EMPTY), (li - 1) & 1u);
                    if (!ok) break;
                    tc_fence_after();
                    const uint64_t vdesc = vdesc0 + (st * L::TILE) / 16;
#pragma unroll
                    for (int ks = 0; ks < KB / 16; ++ks)
                        umma_bf16_ts(tmem + L::O_COL, tmem + pb * KB + (ks >> 2) * L::P_HALF + (ks & 3) * 8, vdesc + (ks * 16 * 128) / 16, idesc,
                                     ks > 0 || i > 0 ? 1u : 0u);
                    umma_commit(bar(B_V_EMPTY + st));
                    umma_commit(bar(B_PV_DONE + pb));
                }
                if (ok) umma_commit(bar(B_O_FULL));
            }
            umma_commit(bar(B_DRAIN + 1));
            drain(bar(B_DRAIN + 1), 0);
        }
    } else if (E4M3 && warp >= 12) {
        // ---------------------------------------------------------- codes to bf16
        // Warp wc takes 32 keys of a block.  A lane's turn is 16 codes of a key, 16 bytes read and 32 written.  The
        // lanes of a quarter-warp take two keys, one its lower four turns and the other its upper four: reads (rows
        // of 128 bytes) and writes (rows of 128 bytes, 16-byte pieces XOR the key's low bits) then meet no bank twice.
        const int wc = warp - 12;
        bool ok = true;
        uint32_t n = 0, gb = 0;
        for (; w.left > 0 && ok; move_on()) {
            const int seg = w.segment();
            int left = w.keys - w.kb * KB;  // keys behind the block's first that exist
            for (int i = 0; i < seg && ok; ++i, ++gb, left -= KB) {
#pragma unroll 1
                for (int kind = 0; kind < 2 && ok; ++kind, ++n) {  // K, then V
                    const uint32_t st = n % NRAW, to = gb & 1u;
                    ok = wait(bar(B_R_FULL + st), (n / NRAW) & 1u) &&
                         wait(bar((kind ? B_V_EMPTY : B_K_EMPTY) + to), ((gb >> 1) & 1u) ^ 1u);
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) break;
                    const uint32_t src = base + L::RAW_OFF + st * L::RAW, dst = (kind ? sV : sK) + to * L::TILE;
                    constexpr int TURNS = D / 16, AT_ONCE = TURNS < 4 ? TURNS : 4;  // of a key, and in registers
#pragma unroll 1
                    for (int x0 = 0; x0 < TURNS; x0 += AT_ONCE) {
                        uint4 u[AT_ONCE];
                        auto row_of = [&](int x) { return wc * 32 + (D == 128 ? (x >> 1) * 8 : x * 8) + (lane >> 2); };
                        auto piece_of = [&](int x) { return D == 128 ? (lane & 3) + 4 * (((lane >> 2) ^ x) & 1) : lane & 3; };
#pragma unroll
                        for (int y = 0; y < AT_ONCE; ++y) u[y] = ld_shared_v4(src + row_of(x0 + y) * D + piece_of(x0 + y) * 16);
#pragma unroll
                        for (int y = 0; y < AT_ONCE; ++y) {
                            const int row = row_of(x0 + y), c = piece_of(x0 + y);
                            const uint32_t in[4] = {u[y].x, u[y].y, u[y].z, u[y].w};
                            uint32_t out[8];
#pragma unroll
                            for (int e = 0; e < 8; ++e) {
                                const float2 f = e4m3x2_float2(in[e >> 1] >> (16 * (e & 1)));
                                out[e] = __byte_perm(__float_as_uint(f.x), __float_as_uint(f.y), 0x7632);  // their upper halves: exact
                            }
                            // Keys of V past the sequence's end are whatever the page holds, and 0 * NaN is NaN.
                            if (kind && row >= left)
#pragma unroll
                                for (int e = 0; e < 8; ++e) out[e] = 0;
                            const uint32_t at = dst + (c >> 2) * BOX + row * 128, piece = (c & 3) * 2, sw = row & 7;
                            st_shared_v4(at + ((piece ^ sw) << 4), out[0], out[1], out[2], out[3]);
                            st_shared_v4(at + (((piece + 1) ^ sw) << 4), out[4], out[5], out[6], out[7]);
                        }
                    }
                    if (kind == 0) {  // 2 x 32 scales a warp; zeros past the sequence's end, where P is 0
                        const bool in = wc * 32 + lane < left;
                        const uint32_t sc = base + L::SC_OFF + (gb % NSC) * (2 * KB * 4) + (wc * 32 + lane) * 4;
                        const uint32_t from = src + L::CODES + (wc * 32 + lane) * 4;
                        st_shared_f32(sc, in ? ld_shared_f32(from) : 0.0f);
                        st_shared_f32(sc + KB * 4, in ? ld_shared_f32(from + KB * 4) : 0.0f);
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(bar(B_R_EMPTY + st));
                        if (kind == 0) mbar_arrive(bar(B_SC_FULL + gb % NSC));
                        mbar_arrive(bar((kind ? B_V_FULL : B_K_FULL) + to));
                    }
                }
            }
        }
    } else if (warp >= 4) {
        // ---------------------------------------------------------- softmax / epilogue
        // Two warps share a TMEM lane quadrant: half hf takes keys [64 hf, 64 hf + 64) of a block and O columns
        // [hf D / 2, + D / 2).  They agree on a row's maximum through shared memory once a block.
        constexpr int KC = KB / 2, DC = L::DC;
        const int q = warp & 3, hf = (warp - 4) >> 2;
        const int r = q * 32 + lane;
        const uint32_t lane_off = static_cast<uint32_t>(q * 32) << 16;
        float* xch = reinterpret_cast<float*>(gbase + L::XCH_OFF);
        Done* done = reinterpret_cast<Done*>(gbase + L::DONE_OFF) + (warp - 4);
        // Failures pass through here before the warps act on them, so the two halves of a quadrant leave together.
        auto pair_all = [&](bool v) -> bool { return named_bar_and(1u + static_cast<uint32_t>(q), 64u, v); };
        bool bad = false;  // a wait gave up: acted on at the next pair_all, with the other half
        // Outputs of a finished segment: O / l as bf16, or O, m and l to the CTA's slot.
        auto epilogue = [&](uint32_t eli) -> bool {
            bool got = !bad && wait(bar(B_O_FULL), eli & 1u);
            got = __all_sync(0xffffffffu, got);
            if (!pair_all(got)) return false;
            tc_fence_after();
            const float l = xch[(4 + (eli & 1) * 2) * QB + r] + xch[(5 + (eli & 1) * 2) * QB + r];
            uint32_t o[DC];
#pragma unroll
            for (int c = 0; c < DC / 32; ++c)
                tmem_ld32(tmem + lane_off + L::O_COL + hf * DC + c * 32, *reinterpret_cast<uint32_t(*)[32]>(&o[c * 32]));
            tmem_ld_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(B_O_EMPTY));
            const Done e = *done;
            if (q * 32 >= e.rows) return true;
            if (e.where >= 0) {
                if (r < e.rows) {
                    const long long at = (static_cast<long long>(blockIdx.x) * 2 + e.where) * QB + r;
                    // In pieces of 16 bytes, [half and quadrant][piece][row of the quadrant]: 512 bytes a store of the
                    // warp (row by row, a part took 3 us more).
                    float4* dst = reinterpret_cast<float4*>(p.part_o + (at - r) * D) + (warp - 4) * (DC / 4) * 32 + lane;
#pragma unroll
                    for (int c = 0; c < DC / 4; ++c)
                        dst[c * 32] = make_float4(__uint_as_float(o[4 * c]), __uint_as_float(o[4 * c + 1]),
                                             __uint_as_float(o[4 * c + 2]), __uint_as_float(o[4 * c + 3]));
                    if (hf == 0) *reinterpret_cast<float2*>(p.part_ml + at * 2) = make_float2(xch[8 * QB + r], l);
                }
                return true;
            }
            const float inv = l != 0.0f ? 1.0f / l : 0.0f;  // nothing seen: zeros
            const int tok = r / p.group;
            __nv_bfloat16* y = p.o + (static_cast<long long>(e.row0 + tok) * p.heads + e.g * p.group + r - tok * p.group) * D + hf * DC;
            // A quadrant of whole tokens, all of them the sequence's, leaves by one TMA store through shared memory
            // (a warp's own 16-byte stores touch 32 lines each); others row by row.
            const bool boxed = !E4M3 && p.o_boxes && q * 32 + 32 <= e.rows;
            constexpr int PIECES = L::STG_ROW / 16;  // 8 or 4
            const uint32_t stg = base + L::STG_OFF + static_cast<uint32_t>((warp - 4) * 32) * L::STG_ROW;
            const uint32_t sw = PIECES == 8 ? lane & 7 : (lane >> 1) & 3;
            if (boxed) {
                if (lane == 0) bulk_wait_group_read0();  // the previous store has read the box
                __syncwarp();
            }
#pragma unroll
            for (int u = 0; u < PIECES; ++u) {
                uint32_t wv[4];
#pragma unroll
                for (int x = 0; x < 4; ++x)
                    wv[x] = pack_bf16x2(__uint_as_float(o[u * 8 + 2 * x]) * inv, __uint_as_float(o[u * 8 + 2 * x + 1]) * inv);
                if (boxed) st_shared_v4(stg + lane * L::STG_ROW + ((u ^ sw) << 4), wv[0], wv[1], wv[2], wv[3]);
                else if (r < e.rows) *reinterpret_cast<uint4*>(y + u * 8) = make_uint4(wv[0], wv[1], wv[2], wv[3]);
            }
            if (boxed) {
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    tma_store_3d(&p.map_o, stg, hf * DC, e.g * p.group, e.row0 + tok);
                    bulk_commit_group();
                }
            }
            return true;
        };
        bool ok = true, pending = false;
        uint32_t gb = 0, li = 0;
        // One turn a segment, and one more for the last one's outputs, so that the epilogue's code is there once.
        for (;; ++li) {
            const bool have = w.left > 0;
            if (!have && !pending) break;
            const int seg = have ? w.segment() : 1;
            const int rows = have ? tile_tokens(w.q, tiling, w.tile) * p.group : 0;
            const bool active = q * 32 < rows;  // some row of the quadrant is the tile's
            // Keys behind the current block's first (lim: that this row sees, from this half's first on; left: that exist).
            int lim = token_keys(w.q, w.keys, w.tile * p.tile_tok + min(r, rows - 1) / p.group) - w.kb * KB - hf * KC;
            int left = w.keys - w.kb * KB;
            float m_ref = -INFINITY, l_sum = 0.0f;
#pragma unroll 1
            for (int i = 0; i < seg; ++i) {
              if (have) {
                const uint32_t st = gb % NS;
                bool got = !bad && wait(bar(B_S_FULL + st), (gb / NS) & 1u);
                // The block with the sequence's last key: rows of V behind it are whatever the page holds, and
                // 0 * NaN is NaN.  They are cleared before P is announced.  This is the only block whose V is waited
                // for here: while the stage's previous block (gb - 2) is still to come, its barrier's parity would
                // read as this one's, so that block's PV comes first (gb - 5's is long done: S of gb needed gb - 3's).
                if (!E4M3 && got && left < KB && left > 0) {
                    const uint32_t vs = gb & 1u;
                    got = (gb < 2 || wait(bar(B_PV_DONE + (gb - 2) % NS), ((gb - 2) / NS) & 1u)) &&
                          wait(bar(B_V_FULL + vs), (gb >> 1) & 1u);
                    if (got) {
                        #pragma unroll 1
                        for (int x = static_cast<int>(threadIdx.x) - 128; x < (KB - left) * NSEG * 8; x += 256) {
                            const int row = left + x / (NSEG * 8), c = x % (NSEG * 8);
                            st_shared_v4(sV + vs * L::TILE + (c >> 3) * BOX + row * 128 + (c & 7) * 16, 0, 0, 0, 0);
                        }
                        fence_proxy_async_smem();
                    }
                }
                if constexpr (E4M3) got = got && wait(bar(B_SC_FULL + gb % NSC), (gb / NSC) & 1u);
                got = __all_sync(0xffffffffu, got);
                constexpr int W = E4M3 ? 32 : KC;  // columns of S in registers at a time
                const uint32_t ts = tmem + lane_off + st * KB + hf * KC;
                uint32_t s[W];
                float mxp = -INFINITY;
                if (got && active) {
                    tc_fence_after();
                    float mx8[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) mx8[e] = -INFINITY;
#pragma unroll
                    for (int c0 = 0; c0 < KC; c0 += W) {
#pragma unroll
                        for (int c = 0; c < W / 32; ++c) tmem_ld32(ts + c0 + c * 32, *reinterpret_cast<uint32_t(*)[32]>(&s[c * 32]));
                        tmem_ld_wait();
                        if constexpr (E4M3) {  // the codes' products times their keys' scales
                            const uint32_t sc = base + L::SC_OFF + (gb % NSC) * (2 * KB * 4) + (hf * KC + c0) * 4;
#pragma unroll
                            for (int c = 0; c < W; c += 4) {
                                const uint4 f = ld_shared_v4(sc + c * 4);
                                float x0, x1, x2, x3;
                                f2_unpack(f2_mul(f2_pack(__uint_as_float(s[c]), __uint_as_float(s[c + 1])),
                                                 f2_pack(__uint_as_float(f.x), __uint_as_float(f.y))), x0, x1);
                                f2_unpack(f2_mul(f2_pack(__uint_as_float(s[c + 2]), __uint_as_float(s[c + 3])),
                                                 f2_pack(__uint_as_float(f.z), __uint_as_float(f.w))), x2, x3);
                                s[c] = __float_as_uint(x0);
                                s[c + 1] = __float_as_uint(x1);
                                s[c + 2] = __float_as_uint(x2);
                                s[c + 3] = __float_as_uint(x3);
                            }
                        }
                        if (lim < c0 + W) {
#pragma unroll
                            for (int c = 0; c < W; ++c)
                                if (c0 + c >= lim) s[c] = __float_as_uint(-INFINITY);
                        }
#pragma unroll
                        for (int c = 0; c < W; c += 16)
#pragma unroll
                            for (int e = 0; e < 8; ++e)
                                mx8[e] = max3(mx8[e], __uint_as_float(s[c + e]), __uint_as_float(s[c + 8 + e]));
                        // 8 bits: half the columns at a time, back to tensor memory for the second pass (with all 64 in
                        // its 128 registers the loop spilled: 3 chunks of 500 tokens over 500 keys took 63 us instead of 55).
                        if constexpr (E4M3) tmem_st32(ts + c0, *reinterpret_cast<const uint32_t(*)[32]>(&s[0]));
                    }
                    if constexpr (E4M3) tmem_st_wait();
                    mxp = max3(max3(mx8[0], mx8[1], mx8[2]), max3(mx8[3], mx8[4], mx8[5]), fmaxf(mx8[6], mx8[7]));
                    xch[((gb & 1) * 2 + hf) * QB + r] = mxp;
                    tc_fence_before();
                }
                // The other half's S is in its registers once this returns, so P may be written over it (8 bits: each half's
                // P goes over its own S).
                if (!pair_all(got)) {
                    ok = false;
                    break;
                }
                if (active) {
                    tc_fence_after();
                    const float mx = fmaxf(mxp, xch[((gb & 1) * 2 + (hf ^ 1)) * QB + r]);
                    const float mxs = mx * p.scale_log2;
                    float alpha = 1.0f;
                    bool rescale = false;
                    if (mxs > m_ref + RESCALE) {
                        alpha = ex2(m_ref - mxs);  // 0 where nothing was seen before
                        m_ref = mxs;
                        rescale = i > 0;
                    }
                    const float ref = m_ref == -INFINITY ? 0.0f : m_ref;
                    const uint64_t scale2 = f2_pack(p.scale_log2, p.scale_log2), neg2 = f2_pack(-ref, -ref);
                    uint64_t acc[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[e] = f2_pack(0.0f, 0.0f);
                    uint32_t pk[KC / 2];
                    const uint32_t vsc = base + L::SC_OFF + (gb % NSC) * (2 * KB * 4) + (KB + hf * KC) * 4;
#pragma unroll
                    for (int c0 = 0; c0 < KC; c0 += W) {
                        if constexpr (E4M3) {
                            tmem_ld32(ts + c0, *reinterpret_cast<uint32_t(*)[32]>(&s[0]));
                            tmem_ld_wait();
                        }
#pragma unroll
                        for (int c = 0; c < W / 2; c += 2) {
                            uint4 vf = make_uint4(0, 0, 0, 0);
                            if constexpr (E4M3) vf = ld_shared_v4(vsc + c0 * 4 + c * 8);
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                float x0, x1;
                                f2_unpack(f2_fma(f2_pack(__uint_as_float(s[2 * (c + h)]), __uint_as_float(s[2 * (c + h) + 1])), scale2, neg2), x0, x1);
                                uint64_t pp = f2_pack(ex2(x0), ex2(x1));
                                acc[(c + h) & 3] = f2_add(acc[(c + h) & 3], pp);
                                if constexpr (E4M3)  // times V's scales
                                    pp = f2_mul(pp, f2_pack(__uint_as_float(h ? vf.z : vf.x), __uint_as_float(h ? vf.w : vf.y)));
                                f2_unpack(pp, x0, x1);
                                pk[c0 / 2 + c + h] = pack_bf16x2(x0, x1);
                            }
                        }
                    }
                    float sum8[8];
#pragma unroll
                    for (int e = 0; e < 4; ++e) f2_unpack(acc[e], sum8[2 * e], sum8[2 * e + 1]);
                    l_sum = l_sum * alpha + (((sum8[0] + sum8[1]) + (sum8[2] + sum8[3])) + ((sum8[4] + sum8[5]) + (sum8[6] + sum8[7])));
                    if (__any_sync(0xffffffffu, rescale)) {
                        // O is rescaled in place: the PV of the previous block must be done.
                        const uint32_t pb = gb - 1;
                        const bool got2 = wait(bar(B_PV_DONE + pb % NS), (pb / NS) & 1u);
                        __syncwarp();
                        if (!__all_sync(0xffffffffu, got2)) {
                            bad = true;
                        } else {
                            tc_fence_after();
#pragma unroll 1
                            for (int c = 0; c < DC / 32; ++c) {
                                uint32_t o[32];
                                const uint32_t ta = tmem + lane_off + L::O_COL + hf * DC + c * 32;
                                tmem_ld32(ta, o);
                                tmem_ld_wait();
#pragma unroll
                                for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
                                tmem_st32(ta, o);
                            }
                            tmem_st_wait();
                        }
                    }
                    // P over the first half of its S buffer: 64 keys as 32 packed columns.
                    tmem_st32(tmem + lane_off + st * KB + hf * L::P_HALF, pk);
                    tmem_st_wait();
                    tc_fence_before();
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(B_P_FULL + st));
                ++gb;
                lim -= KB;
                left -= KB;
              }
                if (i == 0 && pending) {
                    if (!epilogue(li - 1)) {
                        ok = false;
                        break;
                    }
                    pending = false;
                }
            }
            if (!ok || !have) break;
            // The epilogue's pair_all comes before either half reads; by parity, since a segment of one block ends while the
            // other half may still be reading the previous one's.
            xch[(4 + (li & 1) * 2 + hf) * QB + r] = l_sum;
            if (hf == 0) xch[8 * QB + r] = m_ref;
            pending = true;
            __syncwarp();
            if (lane == 0) {
                const bool begins = w.kb == 0, ends = w.kb + seg == w.nkb;
                *done = Done{w.q.row0 + w.tile * p.tile_tok, w.g, rows, begins && ends ? -1 : begins ? 1 : 0};
            }
            move_on();
        }
        if (lane == 0) bulk_wait_group0();  // the stores have left shared memory before the CTA does
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tmem, 512);
}

template <class L>
int launch(const tpi::PagedArgs& a, void* O, void* scratch, bool zero_rest, cudaStream_t stream, std::string* err) {
    Params p;
    memset(&p, 0, sizeof(p));
    const int grid = tpi::device_sm_count();
    p.box_rows = a.page_size;
    int rc;
    if ((rc = tpi::encode_cache(&p.map_k, a, a.K, L::E4M3 ? 0 : 128, p.box_rows, err)) ||
        (rc = tpi::encode_cache(&p.map_v, a, a.V, L::E4M3 ? 0 : 128, p.box_rows, err)))
        return rc;
    p.v = tpi::paged_view(a);
    p.k_scale = a.k_scale;
    p.v_scale = a.v_scale;
    p.o = static_cast<__nv_bfloat16*>(O);
    p.heads = a.heads;
    p.group = a.heads / a.kv_heads;
    p.tile_tok = QB / p.group;
    p.log2_tok = exact_log2(p.tile_tok);
    p.least = a.least;
    p.most = a.most;
    p.kv_per_shard = a.kv_heads / a.t;
    p.shards_per_kv = p.kv_per_shard ? 1 : a.t / a.kv_heads;
    p.scale_log2 = 1.4426950408889634f / sqrtf(static_cast<float>(L::D));
    {
        // Q: the heads of a KV head are G neighbours of one shard, or all heads of t / k neighbouring shards.
        tpi::EncodeTiledFn encode = tpi::encode_fn(err);
        if (!encode) return TP_ERR_CUDA;
        const cuuint64_t hps = static_cast<cuuint64_t>(a.heads / a.t);
        const cuuint64_t dims[4] = {static_cast<cuuint64_t>(L::D), hps, static_cast<cuuint64_t>(a.t),
                                    static_cast<cuuint64_t>(a.tokens)};
        const cuuint64_t strides[3] = {static_cast<cuuint64_t>(L::D) * 2, static_cast<cuuint64_t>(a.shard_w) * 2,
                                       static_cast<cuuint64_t>(a.ld_qkv) * 2};
        const cuuint32_t box[4] = {64, static_cast<cuuint32_t>(p.group / p.shards_per_kv),
                                   static_cast<cuuint32_t>(p.shards_per_kv), static_cast<cuuint32_t>(p.tile_tok)};
        const cuuint32_t estr[4] = {1, 1, 1, 1};
        const CUresult r = encode(&p.map_q, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(a.QKV), dims, strides,
                                  box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
        if (r != CUDA_SUCCESS) {
            if (err) *err = "cuTensorMapEncodeTiled (queries) failed: " + std::to_string(static_cast<int>(r));
            return TP_ERR_CUDA;
        }
    }
    if (32 % p.group == 0) {
        tpi::EncodeTiledFn encode = tpi::encode_fn(err);
        if (!encode) return TP_ERR_CUDA;
        const cuuint64_t dims[3] = {static_cast<cuuint64_t>(L::D), static_cast<cuuint64_t>(a.heads), static_cast<cuuint64_t>(a.tokens)};
        const cuuint64_t strides[2] = {static_cast<cuuint64_t>(L::D) * 2, static_cast<cuuint64_t>(L::D) * 2 * a.heads};
        const cuuint32_t box[3] = {static_cast<cuuint32_t>(L::DC), static_cast<cuuint32_t>(p.group), static_cast<cuuint32_t>(32 / p.group)};
        const cuuint32_t estr[3] = {1, 1, 1};
        const CUresult r = encode(&p.map_o, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, O, dims, strides, box, estr,
                                  CU_TENSOR_MAP_INTERLEAVE_NONE,
                                  L::STG_ROW == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                                  CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
        if (r != CUDA_SUCCESS) {
            if (err) *err = "cuTensorMapEncodeTiled (outputs) failed: " + std::to_string(static_cast<int>(r));
            return TP_ERR_CUDA;
        }
        p.o_boxes = 1;
    }
    const tpi::Scratch s = tpi::scratch_of(grid, QB, L::D);
    uint8_t* w = static_cast<uint8_t*>(scratch);
    p.part_o = reinterpret_cast<float*>(w + s.o);
    p.part_ml = reinterpret_cast<float*>(w + s.ml);
    p.desc = reinterpret_cast<int4*>(w + s.desc);
    p.status = a.status;
    p.timeout_ns = a.timeout_ns;
    static bool configured[64] = {false};
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev < 64 && !configured[dev]) {
        const cudaError_t e = cudaFuncSetAttribute(attn_chunk_kernel<L>, cudaFuncAttributeMaxDynamicSharedMemorySize, L::SMEM);
        if (e != cudaSuccess) return tpi::launched("cudaFuncSetAttribute(chunk attention)", e, err);
        configured[dev] = true;
    }
    rc = tpi::launched("chunk attention launch",
                       tpi::launch_pdl(attn_chunk_kernel<L>, dim3(grid), dim3(L::NT), L::SMEM, stream, p), err);
    if (rc) return rc;
    return tpi::attn_join_launch(a, QB, O, w, s, grid, zero_rest, stream, err);
}

}  // namespace

namespace tpi {

int attn_chunk_launch(const PagedArgs& a, void* O, void* scratch, bool zero_rest, cudaStream_t stream, std::string* err) {
    if (a.head_dim == 128)
        return a.e4m3 ? launch<Lay<128, true>>(a, O, scratch, zero_rest, stream, err)
                      : launch<Lay<128, false>>(a, O, scratch, zero_rest, stream, err);
    return a.e4m3 ? launch<Lay<64, true>>(a, O, scratch, zero_rest, stream, err)
                  : launch<Lay<64, false>>(a, O, scratch, zero_rest, stream, err);
}

}  // namespace tpi
