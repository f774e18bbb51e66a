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
//   warp 0      TMA: Q of a tile as one box {64, heads, shards, tokens}, K and
//               V blocks as one box a page, all lanes issuing; page numbers
//               are read 32 at a time, a window ahead.
//   warp 1      TMEM owner and S issuer: S = Q K^T (tcgen05, fp32) into three
//               TMEM buffers.
//   warp 2      PV issuer: O += P V, P from tensor memory.
//   warps 3..10 softmax, two warps a TMEM lane quadrant, half of a block's keys
//               each; a tile's outputs leave after the next tile's first block,
//               staged in shared memory for whole-line stores.
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
constexpr int NT = 352;          // threads
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
    NUM_BARS = B_DRAIN + 2
};

template <int D_>
struct Lay {
    static constexpr int D = D_;
    static constexpr int NSEG = D / 64;
    static constexpr int TILE = KB * D * 2;  // Q, K or V
    static constexpr int Q_OFF = 0;
    static constexpr int K_OFF = TILE;
    static constexpr int V_OFF = K_OFF + 2 * TILE;
    static constexpr int DC = D / 2;         // O columns of a softmax warp
    static constexpr int STG_ROW = DC * 2;   // bytes of a staged row
    static constexpr int STG_OFF = V_OFF + 2 * TILE;
    static constexpr int XCH_OFF = STG_OFF + 8 * 32 * STG_ROW;  // [3][2][128] fp32
    static constexpr int BAR_OFF = XCH_OFF + 3 * 2 * QB * 4;
    static constexpr int SCAN_OFF = BAR_OFF + 8 * NUM_BARS + 16;
    static constexpr int DATA = SCAN_OFF + 8 * (NT / 32) + 16;
    static constexpr int SMEM = DATA + 1024;
    static constexpr int O_COL = NS * KB;
    static_assert(O_COL + D <= 512 && SMEM <= 232448 && SCAN_OFF % 8 == 0, "configuration");
};

struct Params {
    CUtensorMap map_q;         // the projection buffer as {d, heads a shard, shards, tokens}
    CUtensorMap map_k, map_v;  // the cache as {d, page, k, n_pages}
    PagedView v;
    __nv_bfloat16* o;
    int heads, group, tile_rows, box_rows;
    int kv_per_shard;        // KV heads of a shard, 0 if shards share them
    int shards_per_kv;       // shards that share a KV head (1 if they have their own)
    float scale_log2;
    float* part_o;
    float* part_ml;
    int4* desc;
    unsigned* status;
    unsigned long long timeout_ns;
};

// What the epilogue of a segment needs once its walk has moved on.
struct Done {
    long long row0;  // first row of the sequence
    int g, tile, rows, where;  // where: -1 the output, else the CTA's slot
    float m, l;
    bool bad;
};

template <class L>
__global__ void __launch_bounds__(NT, 1) attn_chunk_kernel(const __grid_constant__ Params p) {
    constexpr int D = L::D, NSEG = L::NSEG;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t* gbase = smem_raw + (base - raw);
    const uint32_t sQ = base + L::Q_OFF, sK = base + L::K_OFF, sV = base + L::V_OFF;
    auto bar = [&](int i) { return base + L::BAR_OFF + 8u * static_cast<uint32_t>(i); };
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(gbase + L::BAR_OFF + 8 * NUM_BARS);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const Tiling tiling = {p.tile_rows, KB, p.group};

    if (threadIdx.x == 0) {
        mbar_init(bar(B_Q_FULL), 1);
        mbar_init(bar(B_Q_EMPTY), 1);
        for (int s = 0; s < 2; ++s) {
            mbar_init(bar(B_K_FULL + s), 1);
            mbar_init(bar(B_K_EMPTY + s), 1);
            mbar_init(bar(B_V_FULL + s), 1);
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
    pdl_trigger();
    pdl_wait();
    const Share share = find_share<NT>(p.v, tiling, gbase + L::SCAN_OFF);  // its barriers cover the set-up above
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    TileWalk w;
    w.start(p.v, tiling, share.s, share.begin - share.seq_begin, share.count);

    if (warp == 0) {
        // ---------------------------------------------------------- TMA producer
        // Order of a segment's loads: for each block i, K(i + 1) then V(i); in
        // place of the K behind the last come the next segment's Q and first K.
        bool ok = true;
        uint32_t q_issued = 0, kn = 0, vn = 0;  // loads issued
        const int log2 = p.v.page_log2, per_block = KB / p.box_rows;
        // Page numbers of a sequence, one a lane: [win, win + 32) and the 32 behind them.
        struct Pages {
            int win, cur, nxt;
        };
        auto page_at = [&](const TileWalk& x, int i) -> int {
            if ((static_cast<long long>(i) << log2) >= x.keys) return -1;
            const int pg = p.v.table[static_cast<long long>(x.s) * p.v.max_pages + i];
            if (pg >= 0 && pg < p.v.n_pages) return pg;
            if (p.status) atomicOr(p.status, kStatusPage);
            return -1;
        };
        auto open = [&](const TileWalk& x) -> Pages {
            const int win = (x.kb * KB) >> log2;
            return Pages{win, page_at(x, win + lane), page_at(x, win + 32 + lane)};
        };
        // K or V of the segment's block i.  A box past the sequence's keys or on no page of the cache has page -1:
        // TMA fills it with zeros.
        auto load_kv = [&](const TileWalk& x, Pages& pg, int i, bool is_v) -> bool {
            uint32_t& n = is_v ? vn : kn;
            const int st = n & 1;
            const uint32_t full = bar((is_v ? B_V_FULL : B_K_FULL) + st), empty = bar((is_v ? B_V_EMPTY : B_K_EMPTY) + st);
            const int key0 = (x.kb + i) * KB, first = key0 >> log2;
            if (first + per_block > pg.win + 32) {  // 32 is a multiple of a block's pages: whole windows
                pg.win += 32;
                pg.cur = pg.nxt;
                pg.nxt = page_at(x, pg.win + 32 + lane);
            }
            bool got = mbar_wait(empty, ((n >> 1) & 1u) ^ 1u, abort_flag, p.status, p.timeout_ns);
            if (!__all_sync(0xffffffffu, got)) return false;
            const int b = lane % per_block, seg = lane / per_block;
            const int key = key0 + b * p.box_rows;
            int page = __shfl_sync(0xffffffffu, pg.cur, ((key >> log2) - pg.win) & 31);
            if (key >= x.keys) page = -1;
            if (lane == 0) mbar_arrive_expect_tx(full, L::TILE);
            __syncwarp();
            if (seg < NSEG)
                tma_load_4d((is_v ? sV : sK) + st * L::TILE + seg * BOX + b * p.box_rows * 128, is_v ? &p.map_v : &p.map_k,
                            full, seg * 64, key & ((1 << log2) - 1), x.g, page);
            __syncwarp();
            ++n;
            return true;
        };
        auto load_q = [&](const TileWalk& x) -> bool {
            bool got = q_issued == 0 || mbar_wait(bar(B_Q_EMPTY), (q_issued - 1) & 1u, abort_flag, p.status, p.timeout_ns);
            if (!__all_sync(0xffffffffu, got)) return false;
            if (lane == 0) {
                mbar_arrive_expect_tx(bar(B_Q_FULL), p.tile_rows * D * 2);
                const int head = p.kv_per_shard ? (x.g % p.kv_per_shard) * p.group : 0;
                const int shard = p.kv_per_shard ? x.g / p.kv_per_shard : x.g * p.shards_per_kv;
                const int token = static_cast<int>(x.q.row0) + x.tile * (p.tile_rows / p.group);
#pragma unroll
                for (int c = 0; c < NSEG; ++c)
                    tma_load_4d(sQ + c * BOX, &p.map_q, bar(B_Q_FULL), 64 * c, head, shard, token);
            }
            __syncwarp();
            ++q_issued;
            return true;
        };
        if (w.left > 0) {
            Pages kp = open(w);
            ok = load_q(w) && load_kv(w, kp, 0, false);
            while (ok && w.left > 0) {
                const int seg = w.segment();
                TileWalk y = w;
                y.next(p.v, tiling);
                Pages vp = open(w), yp{0, -1, -1};
                if (y.left > 0) yp = open(y);
                for (int i = 0; i < seg && ok; ++i) {
                    if (i + 1 < seg) ok = load_kv(w, kp, i + 1, false);
                    else if (y.left > 0) ok = load_q(y) && load_kv(y, yp, 0, false);
                    if (ok) ok = load_kv(w, vp, i, true);
                }
                w = y;
                kp = yp;
            }
        }
        // No copy may be in flight when the CTA's shared memory goes.
        if (q_issued) drain(bar(B_Q_FULL), (q_issued - 1) & 1u);
        for (uint32_t i = kn > 2 ? kn - 2 : 0; i < kn; ++i) drain(bar(B_K_FULL + (i & 1)), (i >> 1) & 1u);
        for (uint32_t i = vn > 2 ? vn - 2 : 0; i < vn; ++i) drain(bar(B_V_FULL + (i & 1)), (i >> 1) & 1u);
    } else if (warp == 1) {
        // ---------------------------------------------------------- S issuer
        if (lane == 0) {
            constexpr uint32_t idesc = idesc_bf16_f32(QB, KB);
            const uint64_t qdesc = sdesc_sw128(sQ), kdesc0 = sdesc_sw128(sK);
            bool ok = true;
            uint32_t gb = 0, li = 0;
            for (; w.left > 0 && ok; w.next(p.v, tiling), ++li) {
                const int seg = w.segment();
                ok = mbar_wait(bar(B_Q_FULL), li & 1u, abort_flag, p.status, p.timeout_ns);
                for (int i = 0; i < seg && ok; ++i, ++gb) {
                    const uint32_t st = gb & 1u, sb = gb % NS;
                    // Buffer sb held P of block gb - NS: its PV must have read it.
                    ok = (gb < NS || mbar_wait(bar(B_PV_DONE + sb), ((gb - NS) / NS) & 1u, abort_flag, p.status,
                                               p.timeout_ns)) &&
                         mbar_wait(bar(B_K_FULL + st), (gb >> 1) & 1u, abort_flag, p.status, p.timeout_ns);
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
                    ok = mbar_wait(bar(B_P_FULL + pb), (gb / NS) & 1u, abort_flag, p.status, p.timeout_ns) &&
                         mbar_wait(bar(B_V_FULL + st), (gb >> 1) & 1u, abort_flag, p.status, p.timeout_ns);
                    // The first PV of a segment overwrites O: the previous epilogue must have read it.
                    if (ok && i == 0 && li > 0)
                        ok = mbar_wait(bar(B_O_EMPTY), (li - 1) & 1u, abort_flag, p.status, p.timeout_ns);
                    if (!ok) break;
                    tc_fence_after();
                    const uint64_t vdesc = vdesc0 + (st * L::TILE) / 16;
#pragma unroll
                    for (int ks = 0; ks < KB / 16; ++ks)
                        umma_bf16_ts(tmem + L::O_COL, tmem + pb * KB + ks * 8, vdesc + (ks * 16 * 128) / 16, idesc,
                                     ks > 0 || i > 0 ? 1u : 0u);
                    umma_commit(bar(B_V_EMPTY + st));
                    umma_commit(bar(B_PV_DONE + pb));
                }
                if (ok) umma_commit(bar(B_O_FULL));
            }
            umma_commit(bar(B_DRAIN + 1));
            drain(bar(B_DRAIN + 1), 0);
        }
    } else {
        // ---------------------------------------------------------- softmax / epilogue
        // Two warps share a TMEM lane quadrant: half hf takes keys [64 hf, 64 hf + 64) of a block and O columns
        // [hf D / 2, + D / 2).  They agree on a row's maximum through shared memory once a block.
        constexpr int KC = KB / 2, DC = L::DC;
        const int q = warp & 3, hf = (warp - 3) >> 2;
        const int r = q * 32 + lane;
        const uint32_t lane_off = static_cast<uint32_t>(q * 32) << 16;
        float* xch = reinterpret_cast<float*>(gbase + L::XCH_OFF);
        if (threadIdx.x == 96) p.desc[blockIdx.x] = make_int4(0, 0, 0, 0);
        // Failures pass through here before the warps act on them, so the two halves of a quadrant leave together.
        auto pair_all = [&](bool v) -> bool { return named_bar_and(1u + static_cast<uint32_t>(q), 64u, v); };
        // Outputs of a finished segment: O / l as bf16, or O, m and l to the CTA's slot.
        auto epilogue = [&](const Done& e, uint32_t eli) -> bool {
            bool got = !e.bad && mbar_wait(bar(B_O_FULL), eli & 1u, abort_flag, p.status, p.timeout_ns);
            got = __all_sync(0xffffffffu, got);
            xch[4 * QB + hf * QB + r] = e.l;
            if (!pair_all(got)) return false;
            tc_fence_after();
            const float l = xch[4 * QB + r] + xch[5 * QB + r];
            uint32_t o[DC];
#pragma unroll
            for (int c = 0; c < DC / 32; ++c)
                tmem_ld32(tmem + lane_off + L::O_COL + hf * DC + c * 32, *reinterpret_cast<uint32_t(*)[32]>(&o[c * 32]));
            tmem_ld_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(B_O_EMPTY));
            if (q * 32 >= e.rows) return true;
            if (e.where >= 0) {
                if (r < e.rows) {
                    const long long at = (static_cast<long long>(blockIdx.x) * 2 + e.where) * QB + r;
                    float4* dst = reinterpret_cast<float4*>(p.part_o + at * D + hf * DC);
#pragma unroll
                    for (int c = 0; c < DC / 4; ++c)
                        dst[c] = make_float4(__uint_as_float(o[4 * c]), __uint_as_float(o[4 * c + 1]),
                                             __uint_as_float(o[4 * c + 2]), __uint_as_float(o[4 * c + 3]));
                    if (hf == 0) *reinterpret_cast<float2*>(p.part_ml + at * 2) = make_float2(e.m, l);
                }
                return true;
            }
            // Rows through shared memory, so that neighbouring lanes store neighbouring pieces of a row.
            const float inv = l != 0.0f ? 1.0f / l : 0.0f;  // nothing seen: zeros
            constexpr int PIECES = L::STG_ROW / 16;          // 8 or 4
            const uint32_t stg = base + L::STG_OFF + static_cast<uint32_t>((warp - 3) * 32) * L::STG_ROW;
            auto at = [&](uint32_t row, uint32_t u) {
                const uint32_t x = PIECES == 8 ? row & 7u : (row >> 1) & 3u;
                return stg + row * L::STG_ROW + ((u ^ x) << 4);
            };
            __syncwarp();
#pragma unroll
            for (int u = 0; u < PIECES; ++u) {
                uint32_t wv[4];
#pragma unroll
                for (int x = 0; x < 4; ++x)
                    wv[x] = pack_bf16x2(__uint_as_float(o[u * 8 + 2 * x]) * inv, __uint_as_float(o[u * 8 + 2 * x + 1]) * inv);
                st_shared_v4(at(lane, u), wv[0], wv[1], wv[2], wv[3]);
            }
            __syncwarp();
            constexpr int STEP = 32 / PIECES;
#pragma unroll
            for (int i = 0; i < 32 / STEP; ++i) {
                const int row = i * STEP + lane / PIECES, u = lane % PIECES;
                const uint4 x = ld_shared_v4(at(row, u));
                if (q * 32 + row < e.rows) {
                    const unsigned rr = static_cast<unsigned>(e.tile * p.tile_rows + q * 32 + row), grp = p.group;
                    const long long token = e.row0 + rr / grp;
                    __nv_bfloat16* y = p.o + (token * p.heads + e.g * p.group + rr % grp) * D + hf * DC + u * 8;
                    *reinterpret_cast<uint4*>(y) = x;
                }
            }
            return true;
        };
        bool ok = true, pending = false;
        Done pd{};
        uint32_t gb = 0, li = 0;
        for (; w.left > 0; w.next(p.v, tiling), ++li) {
            const int seg = w.segment();
            Done cur;
            cur.row0 = w.q.row0;
            cur.g = w.g;
            cur.tile = w.tile;
            cur.rows = static_cast<int>(pmin(p.tile_rows, static_cast<long long>(w.q.n) * p.group -
                                                              static_cast<long long>(w.tile) * p.tile_rows));
            const bool begins = w.kb == 0, ends = w.kb + seg == w.nkb;
            cur.where = begins && ends ? -1 : begins ? 1 : 0;
            if (begins && !ends && threadIdx.x == 96) {
                const long long first = share.begin + share.count - seg;
                const int last = static_cast<int>((first + w.nkb - 1) / share.per);
                p.desc[blockIdx.x] = make_int4(w.s, w.g, w.tile, last - static_cast<int>(blockIdx.x) + 1);
            }
            const bool active = q * 32 < cur.rows;  // some row of the quadrant is the tile's
            const int seen = r < cur.rows ? row_keys(w.q, w.keys, static_cast<long long>(w.tile) * p.tile_rows + r, p.group) : 0;
            float m_ref = -INFINITY, l_sum = 0.0f;
            bool bad = false;
            for (int i = 0; i < seg; ++i, ++gb) {
                const uint32_t st = gb % NS;
                const int key0 = (w.kb + i) * KB;
                bool got = !bad && mbar_wait(bar(B_S_FULL + st), (gb / NS) & 1u, abort_flag, p.status, p.timeout_ns);
                // The block with the sequence's last key: rows of V behind it are whatever the page holds, and
                // 0 * NaN is NaN.  They are cleared before P is announced.
                if (got && key0 + KB > w.keys && key0 < w.keys) {
                    const uint32_t vs = gb & 1u;
                    got = mbar_wait(bar(B_V_FULL + vs), (gb >> 1) & 1u, abort_flag, p.status, p.timeout_ns);
                    if (got) {
                        const int from = w.keys - key0;
                        for (int x = static_cast<int>(threadIdx.x) - 96; x < (KB - from) * NSEG * 8; x += 256) {
                            const int row = from + x / (NSEG * 8), c = x % (NSEG * 8);
                            st_shared_v4(sV + vs * L::TILE + (c >> 3) * BOX + row * 128 + (c & 7) * 16, 0, 0, 0, 0);
                        }
                        fence_proxy_async_smem();
                    }
                }
                got = __all_sync(0xffffffffu, got);
                uint32_t s[KC];
                float mxp = -INFINITY;
                if (got && active) {
                    tc_fence_after();
#pragma unroll
                    for (int c = 0; c < KC / 32; ++c)
                        tmem_ld32(tmem + lane_off + st * KB + hf * KC + c * 32, *reinterpret_cast<uint32_t(*)[32]>(&s[c * 32]));
                    tmem_ld_wait();
                    const int lim = seen - (key0 + hf * KC);  // columns that the row sees
                    if (lim < KC) {
#pragma unroll
                        for (int c = 0; c < KC; ++c)
                            if (c >= lim) s[c] = __float_as_uint(-INFINITY);
                    }
                    float mx8[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) mx8[e] = fmaxf(__uint_as_float(s[e]), __uint_as_float(s[8 + e]));
#pragma unroll
                    for (int c = 16; c < KC; c += 16)
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            mx8[e] = max3(mx8[e], __uint_as_float(s[c + e]), __uint_as_float(s[c + 8 + e]));
                    mxp = max3(max3(mx8[0], mx8[1], mx8[2]), max3(mx8[3], mx8[4], mx8[5]), fmaxf(mx8[6], mx8[7]));
                    xch[((gb & 1) * 2 + hf) * QB + r] = mxp;
                    tc_fence_before();
                }
                // The other half's S is in its registers once this returns, so P may be written over it.
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
#pragma unroll
                    for (int c = 0; c < KC / 2; ++c) {
                        float x0, x1;
                        f2_unpack(f2_fma(f2_pack(__uint_as_float(s[2 * c]), __uint_as_float(s[2 * c + 1])), scale2, neg2), x0, x1);
                        const float p0 = ex2(x0), p1 = ex2(x1);
                        acc[c & 3] = f2_add(acc[c & 3], f2_pack(p0, p1));
                        pk[c] = pack_bf16x2(p0, p1);
                    }
                    float sum8[8];
#pragma unroll
                    for (int e = 0; e < 4; ++e) f2_unpack(acc[e], sum8[2 * e], sum8[2 * e + 1]);
                    l_sum = l_sum * alpha + (((sum8[0] + sum8[1]) + (sum8[2] + sum8[3])) + ((sum8[4] + sum8[5]) + (sum8[6] + sum8[7])));
                    if (__any_sync(0xffffffffu, rescale)) {
                        // O is rescaled in place: the PV of the previous block must be done.
                        const uint32_t pb = gb - 1;
                        const bool got2 = mbar_wait(bar(B_PV_DONE + pb % NS), (pb / NS) & 1u, abort_flag, p.status, p.timeout_ns);
                        __syncwarp();
                        if (!__all_sync(0xffffffffu, got2)) {
                            bad = true;  // acted on at the next pair_all, with the other half
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
                    tmem_st32(tmem + lane_off + st * KB + hf * (KC / 2), pk);
                    tmem_st_wait();
                    tc_fence_before();
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(B_P_FULL + st));
                if (i == 0 && pending) {
                    if (!epilogue(pd, li - 1)) {
                        ok = false;
                        break;
                    }
                    pending = false;
                }
            }
            if (!ok) break;
            cur.m = m_ref;
            cur.l = l_sum;
            cur.bad = bad;
            pd = cur;
            pending = true;
        }
        if (ok && pending) epilogue(pd, li - 1);
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
    if ((rc = tpi::encode_cache(&p.map_k, a, a.K, 128, p.box_rows, err)) ||
        (rc = tpi::encode_cache(&p.map_v, a, a.V, 128, p.box_rows, err)))
        return rc;
    p.v = tpi::paged_view(a);
    p.o = static_cast<__nv_bfloat16*>(O);
    p.heads = a.heads;
    p.group = a.heads / a.kv_heads;
    p.tile_rows = QB / p.group * p.group;
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
                                   static_cast<cuuint32_t>(p.shards_per_kv), static_cast<cuuint32_t>(QB / p.group)};
        const cuuint32_t estr[4] = {1, 1, 1, 1};
        const CUresult r = encode(&p.map_q, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(a.QKV), dims, strides,
                                  box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
        if (r != CUDA_SUCCESS) {
            if (err) *err = "cuTensorMapEncodeTiled (queries) failed: " + std::to_string(static_cast<int>(r));
            return TP_ERR_CUDA;
        }
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
                       tpi::launch_pdl(attn_chunk_kernel<L>, dim3(grid), dim3(NT), L::SMEM, stream, p), err);
    if (rc) return rc;
    return tpi::attn_join_launch(a, p.tile_rows, QB, O, w, s, grid, zero_rest, stream, err);
}

}  // namespace

namespace tpi {

int attn_chunk_launch(const PagedArgs& a, void* O, void* scratch, bool zero_rest, cudaStream_t stream, std::string* err) {
    return a.head_dim == 128 ? launch<Lay<128>>(a, O, scratch, zero_rest, stream, err)
                             : launch<Lay<64>>(a, O, scratch, zero_rest, stream, err);
}

}  // namespace tpi
