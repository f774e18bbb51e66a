// tp_attn_paged.cu -- causal GQA attention of new tokens over a paged
// key/value cache: the kernel for few query rows per sequence and KV head
// (single tokens, drafts), and the joining of split work.
//
// For query head j of a token at position p, with KV head g = j / (a/k):
//   O = sum_{p' <= p} 2^{x_p' - m} V[p'] / sum_{p' <= p} 2^{x_p' - m},
//   x_p' = Q . K[p'] log2(e) / sqrt d,   m a running maximum,
// one pass over the keys.  An 8-bit cache holds K[p'] = kc[p'] ks[p'] and
// V[p'] = vc[p'] vs[p'] (codes and a scale a token): the scales stay outside
// the products,
//   x_p' = (Q . kc[p']) ks[p'] log2(e) / sqrt d,   sum 2^{x - m} vs vc.
//
// With G = a/k query rows per token and KV head, every key read from memory is
// used by a few rows only, so the cache's bytes bound the kernel (16 rows a
// tile: 16 multiply-adds a byte, a few per cent of the tensor cores' rate).
// The work is cut into equal shares of key blocks (tp_paged_index.h), one
// persistent CTA an SM:
//   warps 8, 9  producers of K and of V: TMA boxes of one page each into a ring
//               of key blocks; page numbers are read 32 at a time and ahead.
//   warps 0..7  consumers, 16 or 32 keys of a block each: S^T = K Q^T and
//               O^T += V^T P^T by mma.sync m16n8k16, a running maximum of their
//               own; at a tile's end the eight are merged in shared memory.
// The keys (and d) are the products' 16 rows and the query rows their 8 columns:
// single tokens of 8 heads or fewer then waste no half of a product, which
// matters at mma.sync's 1000 multiply-adds a clock and SM.  P^T goes from S^T's
// registers to the second product's operand by movmatrix.  mma.sync rather than
// tcgen05, whose tile has 64 rows at least and whose P makes a round trip
// through tensor memory.  P is rounded to V's type for that product, whose operands
// have one type: to bf16, at most 2^-8 of each weight, at random (outputs off by
// 0.0023 of their size where one rounding at the end gives 0.0017), or beside codes
// to fp16, 2^-11 (0.0017).  Sums, maxima and O are fp32.
//
// Measured, 32 query heads on 8 KV heads of 128: 64 single tokens over 500 to
// 16000 keys from bf16 (1.04 GB) 160 us, 6.5 TB/s or 0.96 of the copy rate; over
// 1000 to 32000 keys from 8 bits (1.17 GB) 203 us, 5.7 TB/s or 0.85: twice the keys a
// byte and the codes' conversion to fp16 make a block's chain of dependent steps as
// long as its loads (45% of the issue slots used, 15% of the matrix pipe).  One token
// over 4096 keys 10.9 us: two launches, the look-up of the shares and one block a
// CTA, each at its latency.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstring>
#include <string>

#include "tp_attn_paged.cuh"

namespace {

using namespace tpk;
using tpi::launched;
using tpi::Scratch;

constexpr int R = 16;        // query rows of a tile, at most (8 for NB = 1): rows of a slot
constexpr float RESCALE = 8.0f;  // log2 of the growth of a weight before the sums are rescaled

// Head dimension, element type, eights of query rows, consumer warps, those that share a key block
// (the NW / WPB sets of warps take blocks in turn), groups of 16 keys that a warp
// takes of a block, ring stages.
template <int D_, bool E4M3_, int NB_, int NW_, int WPB_, int NG_, int NST_>
struct Cfg {
    static constexpr int D = D_, NB = NB_, NW = NW_, WPB = WPB_, NG = NG_, NST = NST_;
    static constexpr int NT = 32 * (NW + 2);
    static constexpr bool E4M3 = E4M3_;
    static constexpr int LOG2_KB = WPB * NG == 8 ? 7 : 6;
    static constexpr int KB = 1 << LOG2_KB;
    static_assert(KB == 16 * WPB * NG, "keys of a block");
    static constexpr int ROW = E4M3 ? D : 2 * D;       // bytes of a cached row
    static constexpr int SEG = ROW < 128 ? ROW : 128;  // bytes of a TMA box row (one swizzle span)
    static constexpr int NSEG = ROW / SEG;
    static constexpr int TILE = KB * ROW;              // bytes of K (or V) of a block
    static constexpr int SCALES = E4M3 ? 2 * KB * 4 : 0;
    static constexpr int STAGE = 2 * TILE;
    static constexpr int SC_OFF = NST * STAGE;
    static constexpr int ACC_OFF = SC_OFF + NST * SCALES;
    static constexpr int LD_ACC = D + 4;               // floats; 16-byte rows, shifted banks
    static constexpr int XM_OFF = ACC_OFF + NW * 8 * LD_ACC * 4;  // 8 rows of a tile at a time
    static constexpr int BAR_OFF = XM_OFF + 3 * NW * R * 4;
    static constexpr int SCAN_OFF = BAR_OFF + 8 * 2 * NST;
    static constexpr int WALK_OFF = SCAN_OFF + 8 * (NW + 4);  // one walk a warp, and the producers' ahead
    static constexpr int PAGE_OFF = WALK_OFF + (NW + 4) * sizeof(TileWalk);  // page numbers of the two producers
    static constexpr int DATA = PAGE_OFF + 2 * 64 * 4;
    static constexpr int SMEM = DATA + 1024;
    static_assert(SMEM <= 232448, "shared memory");
    // A set of warps that met a stage every second time only could find its barrier two phases behind, which
    // reads as done.
    static_assert(NST % (NW / WPB) == 0, "every stage belongs to one set of warps");
};

struct Params {
    CUtensorMap map_k, map_v;  // the cache as {d, page, k, n_pages}, box {SEG, min(page, KB), 1, 1}
    PagedView v;
    const float *k_scale, *v_scale;
    const __nv_bfloat16* qkv;
    long long ld_qkv;
    __nv_bfloat16* o;
    int heads, heads_per_shard, shard_w, group, tile_tok, log2_tok, box_rows, least, most;
    float scale_log2;
    float* part_o;   // [grid][2][R][D], rows as they are
    float* part_ml;  // [grid][2][R][2]
    int4* desc;      // [grid]: first row, KV head, rows, parts of the tile that begins in a CTA's slot 1
    unsigned* status;
    unsigned long long timeout_ns;
};

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

template <bool F16>
__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if constexpr (F16)
        asm(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%0, %1, %2, %3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%0, %1, %2, %3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Transposes an 8 x 8 matrix of 16-bit elements, two neighbours of a row a lane.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}

// Byte offset of 16-byte piece c of row r in a box of SEG-byte rows written
// by TMA with the swizzle of that span: 128 bytes XOR the row's 8 with the
// piece, 64 bytes two rows to a 128-byte line.
template <int SEG>
__device__ __forceinline__ uint32_t swz(uint32_t r, uint32_t c) {
    if constexpr (SEG == 128) return r * 128 + ((c ^ (r & 7)) << 4);
    else return r * 64 + ((c ^ ((r >> 1) & 3)) << 4);
}

template <class C>
__global__ void __launch_bounds__(C::NT, 1) attn_few_kernel(const __grid_constant__ Params p) {
    constexpr int D = C::D, KB = C::KB, NST = C::NST, NG = C::NG, NW = C::NW, NB = C::NB;
    constexpr bool E4M3 = C::E4M3;
    extern __shared__ uint8_t smem_raw[];
    __shared__ int abort_word;
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t* gbase = smem_raw + (base - raw);
    const uint32_t full0 = base + C::BAR_OFF, empty0 = full0 + 8 * NST;
    volatile int* abort_flag = &abort_word;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const Tiling tiling = {p.tile_tok, p.group, C::LOG2_KB, p.log2_tok, p.least, p.most};
    const Waiter wait = {abort_flag, p.status, p.timeout_ns};

    if (threadIdx.x == 0) {
        for (int i = 0; i < NST; ++i) {
            mbar_init(full0 + 8 * i, E4M3 ? 2 + 2 * (KB / 4) : 2);  // the two producers, and their lanes that copy scales
            mbar_init(empty0 + 8 * i, C::WPB);
        }
        abort_word = 0;
        fence_barrier_init();
        tma_prefetch_desc(&p.map_k);
        tma_prefetch_desc(&p.map_v);
    }
    __syncthreads();
    pdl_trigger();
    pdl_wait();
    TileWalk* walks = reinterpret_cast<TileWalk*>(gbase + C::WALK_OFF);
    TileWalk& w = walks[warp];  // each warp walks on its own, in shared memory; lane 0 moves
    const Share share = find_share<C::NT>(p.v, tiling, reinterpret_cast<long long*>(gbase + C::SCAN_OFF), w);
    auto move_on = [&] {
        __syncwarp();
        if (lane == 0) w.next(p.v, tiling);
        __syncwarp();
    };

    if (warp >= NW) {
        // ------------------------------------------------------ producers: K, V
        const bool is_v = warp > NW;
        const int log2 = p.v.page_log2, page_mask = (1 << log2) - 1, per_block = KB / p.box_rows;
        const int box_log2 = log2 < C::LOG2_KB ? log2 : C::LOG2_KB;
        const CUtensorMap* map = is_v ? &p.map_v : &p.map_k;
        const float* scales = is_v ? p.v_scale : p.k_scale;
        // Page numbers of two windows of 32 pages: page i of the sequence at ring[i - first page of the segment, mod 64].
        int* ring = reinterpret_cast<int*>(gbase + C::PAGE_OFF) + (is_v ? 64 : 0);
        // Page i of a segment's sequence; -1: past its keys, or on no page of the cache (TMA fills such a box with
        // zeros and reads nothing).
        auto page_at = [&](const TileWalk& x, int i) -> int {
            if ((static_cast<long long>(i) << log2) >= x.keys) return -1;
            const int pg = p.v.table[static_cast<long long>(x.s) * p.v.max_pages + i];
            if (pg >= 0 && pg < p.v.n_pages) return pg;
            if (p.status) atomicOr(p.status, kStatusPage);
            return -1;
        };
        // y walks a segment ahead: the first pages of the next segment are read in time.
        TileWalk& y = walks[NW + 2 + (is_v ? 1 : 0)];
        if (lane == 0) y = w;
        __syncwarp();
        int first = -1, behind = -1, n = 0;  // n: blocks issued
        if (y.left > 0) {
            first = page_at(y, ((y.kb * KB) >> log2) + lane);
            behind = page_at(y, ((y.kb * KB) >> log2) + 32 + lane);
        }
        bool ok = true;
        while (y.left > 0 && ok) {
            __syncwarp();
            if (lane == 0) {
                w = y;
                y.next(p.v, tiling);
            }
            __syncwarp();
            const int seg = w.segment(), g = w.g, page0 = (w.kb * KB) >> log2;
            int next = behind, key0 = w.kb * KB, done = 0;  // done: first page of the window's first block
            ring[lane] = first;
            __syncwarp();
            if (y.left > 0) {
                first = page_at(y, ((y.kb * KB) >> log2) + lane);
                behind = page_at(y, ((y.kb * KB) >> log2) + 32 + lane);
            }
            ring[32 + lane] = next;
            next = page_at(w, page0 + 64 + lane);
            __syncwarp();
            for (int i = 0; i < seg; ++i, ++n, key0 += KB) {
                const int at = (key0 >> log2) - page0;  // the block's first page
                if (at - done >= 32) {                  // a window is behind: the next but one takes its place
                    done += 32;
                    ring[(done + 32 + lane) & 63] = next;
                    next = page_at(w, page0 + done + 64 + lane);
                    __syncwarp();
                }
                const int st = n % NST;
                const uint32_t full = full0 + 8 * st;
                ok = __all_sync(0xffffffffu, wait(empty0 + 8 * st, ((n / NST) & 1) ^ 1));
                if (!ok) break;
                const uint32_t dst = base + st * C::STAGE + (is_v ? C::TILE : 0);
                const uint32_t sc = base + C::SC_OFF + st * C::SCALES + (is_v ? KB * 4 : 0);
                if constexpr (E4M3) {
                    // The block's scales, four keys a lane (of one page: it has 16 keys at least); those of no page are zeros.
                    // A copy a page, by the thread that issues the boxes, cost 48 single tokens over 8000 keys 265 us
                    // at 16 keys a page and 172 at 32, where this takes 173 and 138 (131 at 128).
                    static_assert(KB == 128, "four keys a lane");
                    const int page = ring[(at + (lane * 4 >> box_log2)) & 63];
                    if (page >= 0) {
                        copy16(sc + lane * 16, scales + paged_row(p.v, page, g, (key0 + lane * 4) & page_mask));
                        copies_arrive(full);
                    } else {
                        st_shared_v4(sc + lane * 16, 0, 0, 0, 0);
                        mbar_arrive(full);
                    }
                }
                if (lane == 0) {
                    mbar_arrive_expect_tx(full, C::TILE);
                    // One lane issues: a copy's operands are uniform registers, so lanes would take turns.
#pragma unroll 1
                    for (int b = 0; b < per_block; ++b) {
                        const int page = ring[(at + b) & 63], off = (key0 + b * p.box_rows) & page_mask;
#pragma unroll
                        for (int c = 0; c < C::NSEG; ++c)
                            tma_load_4d(dst + c * (KB * C::SEG) + b * p.box_rows * C::SEG, map, full, c * (E4M3 ? 128 : 64), off, g, page);
                    }
                }
                __syncwarp();
            }
        }
        // No copy may be in flight when the CTA's shared memory goes.
        if constexpr (E4M3) copies_wait();
        for (int i = max(0, n - NST); i < n; ++i) drain(full0 + 8 * (i % NST), (i / NST) & 1);
    } else {
        // ------------------------------------------------------ consumers
        // Fragments: r0 is a key (or d) of eight, and the query row of the operand Q^T; 2t, 2t + 1 are the query
        // rows of S^T, P^T and O^T that the lane holds.
        const int r0 = lane >> 2, t = lane & 3;
        const int wk = warp % C::WPB;            // the warp's part of a block's keys
        // Maxima in two buffers in turn: a warp may be at its next tile while others still read this one's.
        float* xm = reinterpret_cast<float*>(gbase + C::XM_OFF);
        float* xl = xm + 2 * NW * R;
        float* acc_s = reinterpret_cast<float*>(gbase + C::ACC_OFF);
        bool ok = true;
        int n = 0;
        if (threadIdx.x == 0) p.desc[blockIdx.x] = make_int4(0, 0, 0, 0);
        for (; w.left > 0; move_on()) {
            const int seg = w.segment(), kb0 = w.kb, keys = w.keys, g = w.g;
            const PagedSeq q = w.q;
            const int tok0 = w.tile * p.tile_tok;  // first token of the tile
            const int rows = tile_tokens(q, tiling, w.tile) * p.group;
            // Row i of the tile: its query head's row of the buffer.
            auto q_row = [&](int i) -> const __nv_bfloat16* {
                const int tok = i / p.group, j = g * p.group + i - tok * p.group;
                return p.qkv + static_cast<long long>(q.row0 + tok0 + tok) * p.ld_qkv +
                       static_cast<long long>(j / p.heads_per_shard) * p.shard_w + (j % p.heads_per_shard) * D;
            };
            int lim[NB][2];  // keys that row 8 nb + 2t + e sees
            uint32_t qf[NB][D / 16][2];
            float row_scale[NB][2];
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) {
                const int i = nb * 8 + r0;
                const __nv_bfloat16* x = i < rows ? q_row(i) : nullptr;
                float scale = p.scale_log2;
                if constexpr (!E4M3) {
#pragma unroll
                    for (int ks = 0; ks < D / 16; ++ks) {
                        qf[nb][ks][0] = x ? *reinterpret_cast<const uint32_t*>(x + ks * 16 + 2 * t) : 0u;
                        qf[nb][ks][1] = x ? *reinterpret_cast<const uint32_t*>(x + ks * 16 + 8 + 2 * t) : 0u;
                    }
                } else {
                    // A product may take d in any order that Q and K share: lane t has the 16 codes
                    // 64 hh + 16 t .. + 15 of a key's row in one load, step j of them the four at 4 j.
                    // Q goes to fp16 after a power of two that brings the row's largest value to
                    // [2^14, 2^15): what that pushes under fp16's range is below 2^-38 of the largest.
                    float amax = 0.0f;
                    uint32_t raw4[D / 64][8];
#pragma unroll
                    for (int hh = 0; hh < D / 64; ++hh)
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            const uint4 u = x ? *reinterpret_cast<const uint4*>(x + hh * 64 + t * 16 + c * 8)
                                              : make_uint4(0, 0, 0, 0);
                            raw4[hh][c * 4] = u.x;
                            raw4[hh][c * 4 + 1] = u.y;
                            raw4[hh][c * 4 + 2] = u.z;
                            raw4[hh][c * 4 + 3] = u.w;
                        }
#pragma unroll
                    for (int hh = 0; hh < D / 64; ++hh)
#pragma unroll
                        for (int c = 0; c < 8; ++c) {
                            const float2 f = unpack_bf16x2(raw4[hh][c]);
                            amax = fmaxf(amax, fmaxf(fabsf(f.x), fabsf(f.y)));
                        }
                    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
                    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
                    const int ex = max((__float_as_int(amax) >> 23) - 127, -100);
                    const float down = __int_as_float((127 + 14 - ex) << 23);
                    scale = p.scale_log2 * __int_as_float((127 - 14 + ex) << 23);
#pragma unroll
                    for (int hh = 0; hh < D / 64; ++hh)
#pragma unroll
                        for (int j = 0; j < 4; ++j)
#pragma unroll
                            for (int c = 0; c < 2; ++c) {
                                const float2 f = unpack_bf16x2(raw4[hh][j * 2 + c]);
                                qf[nb][hh * 4 + j][c] = pack_f16x2(f.x * down, f.y * down);
                            }
                }
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int r = nb * 8 + 2 * t + e;
                    lim[nb][e] = r < rows ? token_keys(q, keys, tok0 + r / p.group) : 0;
                    row_scale[nb][e] = __shfl_sync(0xffffffffu, scale, (2 * t + e) * 4);
                }
            }
            // By row: reference and sum; for 8 bits the reference of the weights 2^x vs.
            float m[NB][2], l[NB][2], mv[NB][2], o[NB][D / 16][4];
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    m[nb][e] = mv[nb][e] = -INFINITY;
                    l[nb][e] = 0.0f;
                }
#pragma unroll
                for (int c = 0; c < D / 16; ++c)
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[nb][c][e] = 0.0f;
            }

            for (int i = 0; i < seg; ++i, ++n) {
                if (C::WPB < NW && n % (NW / C::WPB) != warp / C::WPB) continue;
                const int st = n % NST;
                ok = ok && wait(full0 + 8 * st, (n / NST) & 1);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) continue;
                const uint32_t sk = base + st * C::STAGE, sv = sk + C::TILE;
                const int wk0 = wk * (16 * NG), key0 = (kb0 + i) * KB + wk0;  // the warp's keys of the block
                // S^T.  A warp issues in order and a product waits for its accumulator, so neighbouring products go to
                // different ones: CH accumulators of D / CH steps each where there are few keys and rows.
                constexpr int CH = NG * NB >= 4 ? 1 : 4 / (NG * NB) < D / 32 ? 4 / (NG * NB) : D / 32;
                float s[NG][NB][CH][4] = {};
                if constexpr (!E4M3) {
#pragma unroll
                    for (int ks = 0; ks < D / 16; ++ks)
#pragma unroll
                        for (int gr = 0; gr < NG; ++gr) {
                            // Matrices (keys 0-7, 8-15) x (d 0-7, then 8-15) of a step.
                            uint32_t a[4];
                            ldsm4(sk + (ks >> 2) * (KB * 128) + swz<128>(wk0 + gr * 16 + (lane & 15), (ks & 3) * 2 + (lane >> 4)), a);
#pragma unroll
                            for (int nb = 0; nb < NB; ++nb) mma<false>(s[gr][nb][ks % CH], a, qf[nb][ks][0], qf[nb][ks][1]);
                        }
                } else {
#pragma unroll
                    for (int hh = 0; hh < D / 64; ++hh) {
                        uint32_t c[NG][2][4];  // codes of keys r0 and r0 + 8
#pragma unroll
                        for (int x = 0; x < 2 * NG; ++x) {
                            const uint4 u = ld_shared_v4(sk + swz<C::SEG>(wk0 + x * 8 + r0, hh * 4 + t));
                            c[x >> 1][x & 1][0] = u.x;
                            c[x >> 1][x & 1][1] = u.y;
                            c[x >> 1][x & 1][2] = u.z;
                            c[x >> 1][x & 1][3] = u.w;
                        }
#pragma unroll
                        for (int j = 0; j < 4; ++j)
#pragma unroll
                            for (int gr = 0; gr < NG; ++gr) {
                                const uint32_t a[4] = {e4m3x2_f16x2(c[gr][0][j]), e4m3x2_f16x2(c[gr][1][j]),
                                                       e4m3x2_f16x2(c[gr][0][j] >> 16), e4m3x2_f16x2(c[gr][1][j] >> 16)};
#pragma unroll
                                for (int nb = 0; nb < NB; ++nb)
                                    mma<true>(s[gr][nb][j % CH], a, qf[nb][hh * 4 + j][0], qf[nb][hh * 4 + j][1]);
                            }
                    }
                }
                // Scores in the exp2 domain, masked: x[..][2 hk + e] of key r0 + 8 hk and row 2t + e.
                float x[NG][NB][4], lv[NG][2] = {};
#pragma unroll
                for (int gr = 0; gr < NG; ++gr)
#pragma unroll
                    for (int hk = 0; hk < 2; ++hk) {
                        float ks = 1.0f;
                        if constexpr (E4M3) {
                            const float* sc = reinterpret_cast<const float*>(gbase + C::SC_OFF + st * C::SCALES) + wk0 + gr * 16 + hk * 8 + r0;
                            ks = sc[0];
                            lv[gr][hk] = __log2f(sc[KB]);
                        }
                        const int key = key0 + gr * 16 + hk * 8 + r0;
#pragma unroll
                        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                float sum = s[gr][nb][0][2 * hk + e];
#pragma unroll
                                for (int ch = 1; ch < CH; ++ch) sum += s[gr][nb][ch][2 * hk + e];
                                x[gr][nb][2 * hk + e] = key < lim[nb][e] ? sum * (ks * row_scale[nb][e]) : -INFINITY;
                            }
                    }
                uint32_t pb[NG][NB][2];  // P^T as the second product's operand
#pragma unroll
                for (int nb = 0; nb < NB; ++nb) {
                    float pr[NG][4], alpha[2];
                    bool move = false;
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float mx = -INFINITY;
#pragma unroll
                        for (int gr = 0; gr < NG; ++gr) mx = fmaxf(mx, fmaxf(x[gr][nb][e], x[gr][nb][2 + e]));
#pragma unroll
                        for (int f = 4; f < 32; f <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, f));
                        alpha[e] = 1.0f;
                        if (mx > m[nb][e] + RESCALE) {
                            alpha[e] = ex2(m[nb][e] - mx);
                            m[nb][e] = mx;
                            move = true;
                        }
                        const float ref = m[nb][e] == -INFINITY ? 0.0f : m[nb][e];
                        float sum = 0.0f;
#pragma unroll
                        for (int gr = 0; gr < NG; ++gr)
#pragma unroll
                            for (int hk = 0; hk < 2; ++hk) {
                                pr[gr][2 * hk + e] = ex2(x[gr][nb][2 * hk + e] - ref);
                                sum += pr[gr][2 * hk + e];
                            }
                        l[nb][e] = l[nb][e] * alpha[e] + sum;
                    }
                    if constexpr (E4M3) {
                        // Weights 2^(x + log2 vs) against their own largest, which stands for 2^15: fp16's range
                        // whatever the scales.  A weight is rounded to 2^-11 of itself, or to 2^-25 where
                        // it is below fp16's normal range, 2^-40 of the largest.
                        move = false;
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            float y[NG][2], my = -INFINITY;
#pragma unroll
                            for (int gr = 0; gr < NG; ++gr)
#pragma unroll
                                for (int hk = 0; hk < 2; ++hk) {
                                    const float v = x[gr][nb][2 * hk + e];
                                    y[gr][hk] = v == -INFINITY ? v : v + lv[gr][hk];
                                    my = fmaxf(my, y[gr][hk]);
                                }
#pragma unroll
                            for (int f = 4; f < 32; f <<= 1) my = fmaxf(my, __shfl_xor_sync(0xffffffffu, my, f));
                            alpha[e] = 1.0f;
                            if (my > mv[nb][e]) {
                                alpha[e] = ex2(mv[nb][e] - my);
                                mv[nb][e] = my;
                                move = true;
                            }
                            const float rv = (mv[nb][e] == -INFINITY ? 0.0f : mv[nb][e]) - 15.0f;
#pragma unroll
                            for (int gr = 0; gr < NG; ++gr)
#pragma unroll
                                for (int hk = 0; hk < 2; ++hk) pr[gr][2 * hk + e] = ex2(y[gr][hk] - rv);
                        }
                    }
                    if (__any_sync(0xffffffffu, move)) {
#pragma unroll
                        for (int c = 0; c < D / 16; ++c)
#pragma unroll
                            for (int e = 0; e < 4; ++e) o[nb][c][e] *= alpha[e & 1];
                    }
#pragma unroll
                    for (int gr = 0; gr < NG; ++gr)
#pragma unroll
                        for (int hk = 0; hk < 2; ++hk)
                            pb[gr][nb][hk] = transpose8(E4M3 ? pack_f16x2(pr[gr][2 * hk], pr[gr][2 * hk + 1])
                                                             : pack_bf16x2(pr[gr][2 * hk], pr[gr][2 * hk + 1]));
                }
                // O^T += V^T P^T.  Rows of V past the sequence's keys are whatever the page holds: cleared, since
                // 0 * NaN is NaN.  `live` masks the halves of a register that holds keys 2t, 2t + 1 (+ 8).
#pragma unroll
                for (int gr = 0; gr < NG; ++gr) {
                    const int kg = key0 + gr * 16;
                    uint32_t live[2] = {0xffffffffu, 0xffffffffu};
                    const bool tail = kg + 16 > keys;
                    if (tail) {
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const int key = kg + h * 8 + 2 * t;
                            live[h] = (key < keys ? 0xffffu : 0u) | (key + 1 < keys ? 0xffff0000u : 0u);
                        }
                    }
#pragma unroll
                    for (int c0 = 0; c0 < C::ROW / 32; c0 += 2) {
                        // 32 bytes of 16 keys' rows: (keys 0-7, 8-15) x two 16-byte columns, transposed.
                        uint32_t b[2][4];
#pragma unroll
                        for (int y = 0; y < 2; ++y) {
                            const int c = c0 + y;
                            if constexpr (!E4M3)  // keys 0-7: columns 0, 1; keys 8-15: columns 0, 1
                                ldsm4_t(sv + (c >> 2) * (KB * 128) +
                                            swz<128>(wk0 + gr * 16 + (lane & 7) + ((lane >> 4) << 3), (c & 3) * 2 + ((lane >> 3) & 1)), b[y]);
                            else                  // column 0: keys 0-7, 8-15; column 1
                                ldsm4_t(sv + swz<C::SEG>(wk0 + gr * 16 + (lane & 15), c * 2 + (lane >> 4)), b[y]);
                            if (tail) {
                                b[y][0] &= live[0];
                                b[y][1] &= live[E4M3 ? 1 : 0];
                                b[y][2] &= live[E4M3 ? 0 : 1];
                                b[y][3] &= live[1];
                            }
                        }
#pragma unroll
                        for (int y = 0; y < 2; ++y) {
                            if constexpr (!E4M3) {
#pragma unroll
                                for (int nb = 0; nb < NB; ++nb) mma<false>(o[nb][c0 + y], b[y], pb[gr][nb][0], pb[gr][nb][1]);
                            } else {
                                // A 16-bit column is two codes, d and d + 1, a register's halves two keys: even d are
                                // the product's rows 0..7, odd d its rows 8..15.
#pragma unroll
                                for (int h = 0; h < 2; ++h) {
                                    const uint32_t lo = b[y][2 * h], hi = b[y][2 * h + 1];
                                    const uint32_t a[4] = {e4m3x2_f16x2(__byte_perm(lo, 0, 0x0020)), e4m3x2_f16x2(__byte_perm(lo, 0, 0x0031)),
                                                           e4m3x2_f16x2(__byte_perm(hi, 0, 0x0020)), e4m3x2_f16x2(__byte_perm(hi, 0, 0x0031))};
#pragma unroll
                                    for (int nb = 0; nb < NB; ++nb) mma<true>(o[nb][2 * (c0 + y) + h], a, pb[gr][nb][0], pb[gr][nb][1]);
                                }
                            }
                        }
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(empty0 + 8 * st);
            }

            // ---- merge the warps' sums over their keys, 8 rows at a time
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
#pragma unroll
                    for (int f = 4; f < 32; f <<= 1) l[nb][e] += __shfl_xor_sync(0xffffffffu, l[nb][e], f);
                    if (r0 == 0) xm[warp * R + nb * 8 + 2 * t + e] = m[nb][e];
                }
            const bool begins = kb0 == 0, ends = kb0 + seg == w.nkb;
            const int slot = begins ? 1 : 0;
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) {
                if (nb * 8 >= rows) break;
                named_bar_sync(1, 32 * NW);  // the maxima are there, and the previous sums have been read
                float fo[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int r = nb * 8 + 2 * t + e;
                    float mm = -INFINITY;
#pragma unroll
                    for (int y = 0; y < NW; ++y) mm = fmaxf(mm, xm[y * R + r]);
                    // 2^(own reference - common one); the 8-bit cache's weights have a reference of their own.
                    const float f = m[nb][e] == -INFINITY ? 0.0f : ex2(m[nb][e] - mm);
                    fo[e] = f;
                    if constexpr (E4M3) fo[e] = mv[nb][e] == -INFINITY ? 0.0f : ex2(mv[nb][e] - 15.0f - mm);
                    if (r0 == 0) xl[warp * R + r] = l[nb][e] * f;
                }
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float* dst = acc_s + (warp * 8 + 2 * t + e) * C::LD_ACC;
#pragma unroll
                    for (int c = 0; c < D / 16; ++c) {
                        if constexpr (!E4M3) {
                            dst[c * 16 + r0] = o[nb][c][e] * fo[e];
                            dst[c * 16 + 8 + r0] = o[nb][c][2 + e] * fo[e];
                        } else {
                            *reinterpret_cast<float2*>(dst + c * 16 + 2 * r0) = make_float2(o[nb][c][e] * fo[e], o[nb][c][2 + e] * fo[e]);
                        }
                    }
                }
                named_bar_sync(1, 32 * NW);
                if (!ok) continue;
                for (int z = threadIdx.x; z < min(rows - 8 * nb, 8) * (D / 4); z += 32 * NW) {
                    const int ir = z / (D / 4), i = ir + 8 * nb, c = (z % (D / 4)) * 4;
                    float4 a = make_float4(0, 0, 0, 0);
                    float lt = 0.0f, mt = -INFINITY;
#pragma unroll
                    for (int y = 0; y < NW; ++y) {
                        const float4 b = *reinterpret_cast<const float4*>(acc_s + (y * 8 + ir) * C::LD_ACC + c);
                        a.x += b.x;
                        a.y += b.y;
                        a.z += b.z;
                        a.w += b.w;
                        lt += xl[y * R + i];
                        mt = fmaxf(mt, xm[y * R + i]);
                    }
                    if (begins && ends) {
                        const float inv = lt != 0.0f ? 1.0f / lt : 0.0f;  // nothing seen: zeros
                        const int tok = i / p.group;
                        __nv_bfloat16* y = p.o +
                            (static_cast<long long>(q.row0 + tok0 + tok) * p.heads + g * p.group + i - tok * p.group) * D + c;
                        *reinterpret_cast<uint2*>(y) =
                            make_uint2(pack_bf16x2(a.x * inv, a.y * inv), pack_bf16x2(a.z * inv, a.w * inv));
                    } else {
                        const long long at = (static_cast<long long>(blockIdx.x) * 2 + slot) * R + i;
                        *reinterpret_cast<float4*>(p.part_o + at * D + c) = a;
                        if (c == 0) *reinterpret_cast<float2*>(p.part_ml + at * 2) = make_float2(mt, lt);
                    }
                }
            }
            if (begins && !ends && threadIdx.x == 0) {
                // The tile's last block is in CTA (first block + blocks - 1) / per.
                const long long at = share.begin + share.count - seg;
                const int last = share_of(at + w.nkb - 1, share.per);
                p.desc[blockIdx.x] = make_int4(q.row0 + tok0, g, rows, last - static_cast<int>(blockIdx.x) + 1);
            }
            xm = reinterpret_cast<float*>(gbase + C::XM_OFF) + (xm == reinterpret_cast<float*>(gbase + C::XM_OFF) ? NW * R : 0);
        }
    }
    __syncthreads();
}

// Clears the rows of O that no sequence owns.
__device__ __forceinline__ void clear_rest(const PagedView& v, int row_bytes, __nv_bfloat16* o) {
    const int a = imin(imax(v.q_start[0], 0), v.rows), b = imin(imax(v.q_start[v.n_seqs], a), v.rows);
    const long long per = row_bytes / 16, threads = static_cast<long long>(gridDim.x) * blockDim.x;
    const long long me = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x;
    uint4* y = reinterpret_cast<uint4*>(o);
    for (long long i = me; i < a * per; i += threads) y[i] = make_uint4(0, 0, 0, 0);
    for (long long i = b * per + me; i < v.rows * per; i += threads) y[i] = make_uint4(0, 0, 0, 0);
}

// Running (m, l, a) with one more part: O = sum 2^(m_i - m) O_i, l likewise.
// 2^-inf = 0: nothing before, or nothing seen.
__device__ __forceinline__ void join_part(float& m, float& l, float4& a, float2 ml, const float4& b) {
    const float mm = fmaxf(m, ml.x), base = mm == -INFINITY ? 0.0f : mm;
    const float f = ex2(m - base), e = ex2(ml.x - base);
    m = mm;
    l = l * f + ml.y * e;
    a.x = a.x * f + b.x * e;
    a.y = a.y * f + b.y * e;
    a.z = a.z * f + b.z * e;
    a.w = a.w * f + b.w * e;
}
__device__ __forceinline__ uint2 joined(float l, const float4& a) {
    const float inv = l != 0.0f ? 1.0f / l : 0.0f;
    return make_uint2(pack_bf16x2(a.x * inv, a.y * inv), pack_bf16x2(a.z * inv, a.w * inv));
}

// Joins the parts of the tile that begins in slot 1 of CTA blockIdx.x and goes
// on in slot 0 of the next ones, O = sum 2^(m_i - m) O_i / sum 2^(m_i - m) l_i,
// in a fixed order.  Slot 1 of the first CTA is followed in memory by slot 0 of
// the next; then comes every second slot.  Tiles of many rows have few parts: a
// thread takes them one after the other, 16 columns of a row, a warp 32 rows (the
// slots hold 16-byte pieces of 32 rows side by side, so that the chunk kernel's
// stores and these loads are 512 contiguous bytes a warp).  It moves two partial
// tiles a CTA at most (20 MB of fp32, in L2); its time and the parts' stores came
// from 10 to 5 us with that layout (3 chunks of 500 tokens over 500 keys: 40 -> 35 us).
template <int D>
__global__ void __launch_bounds__(1024) attn_join_rows_kernel(PagedView v, int group, int heads, const float* part_o,
                                                              const float* part_ml, const int4* desc, __nv_bfloat16* o,
                                                              int zero_rest) {
    pdl_trigger();
    pdl_wait();
    constexpr int ROWS = 128, HALF = D / 8, QUAD = ROWS / 32;  // pieces of 16 bytes of half a row
    const int4 x = desc[blockIdx.x];  // the tile's first row, KV head, rows, parts
    if (zero_rest) clear_rest(v, heads * D * 2, o);
    const int i = threadIdx.x % ROWS, c = threadIdx.x / ROWS * 4;  // a thread's row, and its first piece of four
    if (i >= x.z || c >= D / 4 || x.w == 0) return;
    float m = -INFINITY, l = 0.0f;
    float4 a[4] = {};
#pragma unroll 2
    for (int k = 0; k < x.w; ++k) {
        const long long slot = static_cast<long long>(blockIdx.x) * 2 + (k == 0 ? 1 : 2 * k);
        const float2 ml = *reinterpret_cast<const float2*>(part_ml + (slot * ROWS + i) * 2);
        const float4* from = reinterpret_cast<const float4*>(part_o + slot * ROWS * D) +
                             (c / HALF * QUAD + i / 32) * HALF * 32 + c % HALF * 32 + i % 32;
        float4 b[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) b[e] = from[e * 32];
        float mm = m, ll = l;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            mm = m;
            ll = l;
            join_part(mm, ll, a[e], ml, b[e]);
        }
        m = mm;
        l = ll;
    }
    const int tok = i / group;
    uint2* y = reinterpret_cast<uint2*>(o + (static_cast<long long>(x.x + tok) * heads + x.y * group + i - tok * group) * D + c * 4);
#pragma unroll
    for (int e = 0; e < 4; e += 2) {
        const uint2 u = joined(l, a[e]), w = joined(l, a[e + 1]);
        *reinterpret_cast<uint4*>(y + e) = make_uint4(u.x, u.y, w.x, w.y);
    }
}

// Tiles of few rows may have a part in every CTA: JW groups of D / 4 lanes a row
// take them in turn (every JW-th), so that one long sequence is not joined at a
// part's latency each (one token over 4096 keys, 32 parts: 13.3 -> 11.5 us for both
// kernels); the groups' sums are joined in order through shared memory.
template <int D>
__global__ void __launch_bounds__(1024) attn_join_parts_kernel(PagedView v, int group, int heads, const float* part_o,
                                                               const float* part_ml, const int4* desc, __nv_bfloat16* o,
                                                               int zero_rest) {
    pdl_trigger();
    pdl_wait();
    constexpr int LANES = D / 4, JW = 8, AT_ONCE = 1024 / LANES / JW;  // rows at once
    __shared__ float4 sums[JW][AT_ONCE][LANES];
    __shared__ float2 mls[JW][AT_ONCE];
    const int4 x = desc[blockIdx.x];  // the tile's first row, KV head, rows, parts
    if (zero_rest) clear_rest(v, heads * D * 2, o);
    const int lane = threadIdx.x % LANES, jw = (threadIdx.x / LANES) % JW, ir = threadIdx.x / (LANES * JW);
    for (int i0 = 0; i0 < x.z; i0 += AT_ONCE) {
        const int i = i0 + ir;
        float m = -INFINITY, l = 0.0f;
        float4 a = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (i < x.z) {
            auto slot = [&](int k) { return (static_cast<long long>(blockIdx.x) * 2 + (k == 0 ? 1 : 2 * k)) * R + i; };
#pragma unroll 4
            for (int k = jw; k < x.w; k += JW)
                join_part(m, l, a, *reinterpret_cast<const float2*>(part_ml + slot(k) * 2),
                          *reinterpret_cast<const float4*>(part_o + slot(k) * D + lane * 4));
        }
        sums[jw][ir][lane] = a;
        if (lane == 0) mls[jw][ir] = make_float2(m, l);
        __syncthreads();
        if (jw == 0 && i < x.z) {
#pragma unroll
            for (int k = 1; k < JW; ++k) join_part(m, l, a, mls[k][ir], sums[k][ir][lane]);
            const int tok = i / group;
            *reinterpret_cast<uint2*>(o + (static_cast<long long>(x.x + tok) * heads + x.y * group + i - tok * group) * D + lane * 4) =
                joined(l, a);
        }
        __syncthreads();
    }
}

template <class C>
int launch_few(const tpi::PagedArgs& a, void* O, void* scratch, bool zero_rest, cudaStream_t stream, std::string* err) {
    Params p;
    memset(&p, 0, sizeof(p));
    const int grid = tpi::device_sm_count();
    p.box_rows = a.page_size < C::KB ? a.page_size : C::KB;
    int rc;
    if ((rc = tpi::encode_cache(&p.map_k, a, a.K, C::SEG, p.box_rows, err)) ||
        (rc = tpi::encode_cache(&p.map_v, a, a.V, C::SEG, p.box_rows, err)))
        return rc;
    p.v = tpi::paged_view(a);
    p.k_scale = a.k_scale;
    p.v_scale = a.v_scale;
    p.qkv = static_cast<const __nv_bfloat16*>(a.QKV);
    p.ld_qkv = a.ld_qkv;
    p.o = static_cast<__nv_bfloat16*>(O);
    p.heads = a.heads;
    p.heads_per_shard = a.heads / a.t;
    p.shard_w = static_cast<int>(a.shard_w);
    p.group = a.heads / a.kv_heads;
    p.tile_tok = 8 * C::NB / p.group;
    p.log2_tok = exact_log2(p.tile_tok);
    p.least = a.least;
    p.most = a.most;
    p.scale_log2 = 1.4426950408889634f / sqrtf(static_cast<float>(C::D));
    const Scratch s = tpi::scratch_of(grid, R, C::D);
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
        const cudaError_t e = cudaFuncSetAttribute(attn_few_kernel<C>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
        if (e != cudaSuccess) return launched("cudaFuncSetAttribute(paged attention)", e, err);
        configured[dev] = true;
    }
    rc = launched("paged attention launch",
                  tpi::launch_pdl(attn_few_kernel<C>, dim3(grid), dim3(C::NT), C::SMEM, stream, p), err);
    if (rc) return rc;
    return tpi::attn_join_launch(a, R, O, w, s, grid, zero_rest, stream, err);
}

template <class Kernel>
cudaError_t join(Kernel kernel, const tpi::PagedArgs& a, void* O, uint8_t* w, const Scratch& s, int grid, bool zero_rest,
                 cudaStream_t stream) {
    return tpi::launch_pdl(kernel, dim3(grid), dim3(1024), 0, stream, tpi::paged_view(a), a.heads / a.kv_heads, a.heads,
                           reinterpret_cast<const float*>(w + s.o), reinterpret_cast<const float*>(w + s.ml),
                           reinterpret_cast<const int4*>(w + s.desc), static_cast<__nv_bfloat16*>(O), zero_rest ? 1 : 0);
}

// Rows of a sequence and KV head that the kernel for few rows is built for.
int few_rows(const tpi::PagedArgs& a) { return a.e4m3 || a.head_dim == 64 ? R : 8; }

// Tiles of 8 rows, or of 16 (not for heads of 128 from bf16).
int few(const tpi::PagedArgs& a, int64_t rows, void* O, void* scratch, bool zero_rest, cudaStream_t stream, std::string* err) {
    if (rows > few_rows(a)) {
        if (err) *err = "paged attention: no kernel for few rows takes " + std::to_string(rows) + " rows of this cache";
        return TP_ERR_UNSUPPORTED;
    }
    if (rows <= 8) {
        if (a.head_dim == 128)
            return a.e4m3 ? launch_few<Cfg<128, true, 1, 8, 4, 2, 4>>(a, O, scratch, zero_rest, stream, err)
                          : launch_few<Cfg<128, false, 1, 8, 4, 1, 4>>(a, O, scratch, zero_rest, stream, err);
        return a.e4m3 ? launch_few<Cfg<64, true, 1, 8, 4, 2, 8>>(a, O, scratch, zero_rest, stream, err)
                      : launch_few<Cfg<64, false, 1, 8, 4, 2, 4>>(a, O, scratch, zero_rest, stream, err);
    }
    if (a.head_dim == 128) return launch_few<Cfg<128, true, 2, 8, 4, 2, 4>>(a, O, scratch, zero_rest, stream, err);
    return a.e4m3 ? launch_few<Cfg<64, true, 2, 8, 4, 2, 8>>(a, O, scratch, zero_rest, stream, err)
                  : launch_few<Cfg<64, false, 2, 8, 4, 2, 4>>(a, O, scratch, zero_rest, stream, err);
}

}  // namespace

namespace tpi {

// The kernel for many rows has the larger tiles.
size_t attn_paged_scratch_bytes(int head_dim) { return scratch_of(device_sm_count(), 128, head_dim).total; }

int attn_join_launch(const PagedArgs& a, int slot_rows, void* O, uint8_t* w, const Scratch& s, int grid,
                     bool zero_rest, cudaStream_t stream, std::string* err) {
    auto kernel = a.head_dim == 128 ? (slot_rows == R ? attn_join_parts_kernel<128> : attn_join_rows_kernel<128>)
                                    : (slot_rows == R ? attn_join_parts_kernel<64> : attn_join_rows_kernel<64>);
    const cudaError_t e = join(kernel, a, O, w, s, grid, zero_rest, stream);
    return launched("paged attention join launch", e, err);
}

int attn_paged_launch(const PagedArgs& a, void* O, void* scratch, bool zero_rest, cudaStream_t stream,
                      std::string* err) {
    if (a.n_seqs == 0) {
        if (!zero_rest) return TP_OK;
        return launched("output reset",
                        cudaMemsetAsync(O, 0, static_cast<size_t>(a.tokens) * a.heads * a.head_dim * 2, stream), err);
    }
    // Few rows a sequence and KV head (the caller's bound on its new tokens, or all rows of the call): one tile
    // of 8 or 16.  More: tiles of 128 on tcgen05.  32 sequences over 1000 / 8000 keys, 8 KV heads, in us:
    //                  bf16 d = 64       e4m3 d = 64       bf16 d = 128      e4m3 d = 128
    //   8 rows   8:    16.0 /  86        19.3 /  81        32.2 / 160        22.6 /  97
    //           16:    18.3 /  88        21.0 /  89        34.6 / 165        30.0 / 134
    //          128:    23.6 / 102        33.6 / 170        33.0 / 162        38.1 / 198
    //  16 rows  16:    21.6 /  91        24.6 /  93        40.0 / 169        35.4 / 140
    //          128:    23.6 / 102        33.7 / 170        33.2 / 164        38.2 / 198
    //  24 rows  16:    30.9 / 165        36.6 / 171        54.2 / 318        55.0 / 260   (two tiles)
    //          128:    23.8 / 103        33.7 / 170        33.7 / 165        38.6 / 199
    const int group = a.heads / a.kv_heads;
    const int64_t most = a.max_new > 0 && a.max_new < a.tokens ? a.max_new : a.tokens;
    if (most * group <= few_rows(a)) return few(a, most * group, O, scratch, zero_rest, stream, err);
    // An 8-bit call that may be a mixture, its mean of new tokens a sequence at most half of the bound on them: a launch
    // of the few-row kernel, which reads codes at the memory's rate, for the sequences of few rows, and one of the
    // 128-row tiles, which take 1.7 us a block whatever their rows, for the others.  One chunk of 500 tokens and 23
    // single ones, one launch and two: over 8000 keys 244 and 186 us, over 2000 80 and 74, over 500 38 and 41 (a table
    // below 1024 keys stays with one).  The host knows no more than that mean.  Where no sequence has few, the empty pair
    // of launches costs 3 to 5 us: 100, 100, 100 and 900 tokens behind 500 keys 49 and 53, behind 8000 263 and 267.
    // So it does where max_new is 0, and all of the call's tokens are the bound: 4 x 500 behind 500 62 and 67, behind
    // 8000 399 and 402; single tokens pay for the empty pair of the 128-row tiles, 32 behind 2000 keys 35 and 40, behind
    // 8000 93 and 99.  From bf16 one launch is faster: 149 and 184 us over 8000.
    if (a.e4m3 && group <= R && 2 * a.tokens <= a.n_seqs * most && static_cast<int64_t>(a.max_pages) * a.page_size >= 1024) {
        const int rows = group <= 8 ? 8 : R;
        PagedArgs part = a;
        part.most = rows / group;
        const int rc = few(part, rows, O, scratch, false, stream, err);
        if (rc) return rc;
        part = a;
        part.least = rows / group + 1;
        return attn_chunk_launch(part, O, scratch, zero_rest, stream, err);
    }
    return attn_chunk_launch(a, O, scratch, zero_rest, stream, err);
}

}  // namespace tpi
