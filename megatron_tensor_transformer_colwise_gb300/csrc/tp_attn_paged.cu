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
//   warp 8      producer: TMA boxes of one page each into a ring of key
//               blocks; the page numbers of 32 pages are read at a time.
//   warps 0..7  consumers, 16 or 32 keys of a block each: S = Q K^T and O += P V by
//               mma.sync m16n8k16 (rows = the tile's 16 query rows, P straight
//               from S's registers), a running maximum of their own; at a
//               tile's end the eight are merged in shared memory.
// mma.sync rather than tcgen05: the tile has 16 rows, tcgen05's least is 64,
// and P would make a round trip through tensor memory.
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

constexpr int R = 16;        // query rows of a tile, at most
constexpr int NW = 8;        // consumer warps
constexpr int NT = 32 * (NW + 1);
constexpr float RESCALE = 8.0f;  // log2 of the growth of a weight before the sums are rescaled

// Head dimension, element type, warps that share a key block (with 4 the two
// halves of the warps take alternate blocks), groups of 16 keys that a warp
// takes of a block, ring stages.
template <int D_, bool E4M3_, int WPB_, int NG_, int NST_>
struct Cfg {
    static constexpr int D = D_, WPB = WPB_, NG = NG_, NST = NST_;
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
    static constexpr int XM_OFF = ACC_OFF + NW * R * LD_ACC * 4;
    static constexpr int BAR_OFF = XM_OFF + 2 * NW * R * 4;
    static constexpr int SCAN_OFF = BAR_OFF + 8 * 2 * NST;
    static constexpr int WALK_OFF = SCAN_OFF + 8 * (NW + 3);  // the share's beginning, then one walk a warp
    static constexpr int DATA = WALK_OFF + (NW + 2) * sizeof(TileWalk);
    static constexpr int SMEM = DATA + 1024;
    static_assert(SMEM <= 232448, "shared memory");
};

struct Params {
    CUtensorMap map_k, map_v;  // the cache as {d, page, k, n_pages}, box {SEG, min(page, KB), 1, 1}
    PagedView v;
    const float *k_scale, *v_scale;
    const __nv_bfloat16* qkv;
    long long ld_qkv;
    __nv_bfloat16* o;
    int heads, heads_per_shard, shard_w, group, tile_tok, log2_tok, box_rows;
    float scale_log2;
    float* part_o;   // [grid][2][R][D]
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
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%0, %1, %2, %3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%0, %1, %2, %3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
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
__global__ void __launch_bounds__(NT, 1) attn_few_kernel(const __grid_constant__ Params p) {
    constexpr int D = C::D, KB = C::KB, NST = C::NST, NG = C::NG;
    constexpr bool E4M3 = C::E4M3;
    extern __shared__ uint8_t smem_raw[];
    __shared__ int abort_word;
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t* gbase = smem_raw + (base - raw);
    const uint32_t full0 = base + C::BAR_OFF, empty0 = full0 + 8 * NST;
    volatile int* abort_flag = &abort_word;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const Tiling tiling = {p.tile_tok, p.group, C::LOG2_KB, p.log2_tok};
    const Waiter wait = {abort_flag, p.status, p.timeout_ns};

    if (threadIdx.x == 0) {
        for (int i = 0; i < NST; ++i) {
            mbar_init(full0 + 8 * i, 1);
            mbar_init(empty0 + 8 * i, C::WPB);
        }
        abort_word = 0;
        fence_barrier_init();
        tma_prefetch_desc(&p.map_k);
        tma_prefetch_desc(&p.map_v);
    }
    pdl_trigger();
    pdl_wait();
    TileWalk* walks = reinterpret_cast<TileWalk*>(gbase + C::WALK_OFF);
    const Share share =  // its barriers cover the set-up above
        find_share<NT>(p.v, tiling, reinterpret_cast<long long*>(gbase + C::SCAN_OFF), walks);
    // Each warp walks on its own, in shared memory; lane 0 moves.
    TileWalk& w = walks[1 + warp];
    if (lane == 0) w = walks[0];
    __syncwarp();
    auto move_on = [&] {
        __syncwarp();
        if (lane == 0) w.next(p.v, tiling);
        __syncwarp();
    };

    if (warp == NW) {
        // ------------------------------------------------------ producer
        bool ok = true;
        int n = 0;  // blocks issued
        for (; w.left > 0 && ok; move_on()) {
            const int seg = w.segment(), kb0 = w.kb, keys = w.keys, g = w.g;
            const int32_t* table = p.v.table + static_cast<long long>(w.s) * p.v.max_pages;
            const int page_rows = 1 << p.v.page_log2;
            const int per_block = KB / p.box_rows;  // boxes (pages, or parts of one) of a block
            int window = -32, held = -1;            // pages [window, window + 32) of the sequence, one a lane
            for (int i = 0; i < seg && ok; ++i, ++n) {
                const int st = n % NST;
                const uint32_t full = full0 + 8 * st;
                const int key0 = (kb0 + i) * KB;
                const int first = key0 >> p.v.page_log2;
                if (first + per_block > window + 32 || first < window) {
                    window = first;
                    const int pg = window + lane;
                    held = -1;
                    if (pg * static_cast<long long>(page_rows) < keys) {
                        held = table[pg];
                        if (held < 0 || held >= p.v.n_pages) {
                            held = -1;
                            if (p.status) atomicOr(p.status, kStatusPage);
                        }
                    }
                }
                ok = wait(empty0 + 8 * st, ((n / NST) & 1) ^ 1);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                // Box b of the block: keys key0 + b * box_rows.  A box past the
                // sequence's keys, or on a page outside the cache, is loaded
                // from page -1: TMA fills it with zeros and reads nothing.
                if constexpr (E4M3) {
                    // Scales, a lane a box; those of no page are zeros.
                    const int k_box = key0 + lane * p.box_rows;
                    int page = __shfl_sync(0xffffffffu, held, (first - window + lane) & 31);
                    if (k_box >= keys) page = -1;
                    const bool mine = lane < per_block;
                    const uint32_t sc = base + C::SC_OFF + st * C::SCALES + lane * p.box_rows * 4;
                    const unsigned scaled = __ballot_sync(0xffffffffu, mine && page >= 0);
                    if (mine && page < 0) {
#pragma unroll 1
                        for (int x = 0; x < p.box_rows; x += 4) {
                            st_shared_v4(sc + x * 4, 0, 0, 0, 0);
                            st_shared_v4(sc + KB * 4 + x * 4, 0, 0, 0, 0);
                        }
                        fence_proxy_async_smem();
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive_expect_tx(full, 2 * C::TILE + 8u * p.box_rows * __popc(scaled));
                } else {
                    if (lane == 0) mbar_arrive_expect_tx(full, 2 * C::TILE);
                }
                // One lane issues: a copy's operands are uniform registers, so lanes would take turns.
#pragma unroll 1
                for (int b = 0; b < per_block; ++b) {
                    const int k_box = key0 + b * p.box_rows, off = k_box & (page_rows - 1);
                    int page = __shfl_sync(0xffffffffu, held, ((k_box >> p.v.page_log2) - window) & 31);
                    if (k_box >= keys) page = -1;
                    if (lane == 0) {
                        const uint32_t dst = base + st * C::STAGE + b * p.box_rows * C::SEG;
#pragma unroll
                        for (int c = 0; c < C::NSEG; ++c) {
                            tma_load_4d(dst + c * (KB * C::SEG), &p.map_k, full, c * (E4M3 ? 128 : 64), off, g, page);
                            tma_load_4d(dst + C::TILE + c * (KB * C::SEG), &p.map_v, full, c * (E4M3 ? 128 : 64), off, g, page);
                        }
                        if (E4M3 && page >= 0) {
                            const uint32_t sc = base + C::SC_OFF + st * C::SCALES + b * p.box_rows * 4;
                            const long long at = paged_row(p.v, page, g, off);
                            bulk_load(sc, p.k_scale + at, p.box_rows * 4, full);
                            bulk_load(sc + KB * 4, p.v_scale + at, p.box_rows * 4, full);
                        }
                    }
                }
                __syncwarp();
            }
        }
        // No copy may be in flight when the CTA's shared memory goes.
        for (int i = max(0, n - NST); i < n; ++i) drain(full0 + 8 * (i % NST), (i / NST) & 1);
    } else {
        // ------------------------------------------------------ consumers
        const int r0 = lane >> 2, t = lane & 3;  // fragment rows r0 and r0 + 8, column pair t
        const int wk = warp % C::WPB;            // the warp's part of a block's keys
        float* xm = reinterpret_cast<float*>(gbase + C::XM_OFF);
        float* xl = xm + NW * R;
        float* acc_s = reinterpret_cast<float*>(gbase + C::ACC_OFF);
        bool ok = true;
        int n = 0;
        if (threadIdx.x == 0) p.desc[blockIdx.x] = make_int4(0, 0, 0, 0);
        for (; w.left > 0; move_on()) {
            const int seg = w.segment(), kb0 = w.kb, keys = w.keys, g = w.g;
            const PagedSeq q = w.q;
            const int tok0 = w.tile * p.tile_tok;  // first token of the tile
            const int rows = tile_tokens(q, tiling, w.tile) * p.group;
            // Row i of the tile: its query head's row of the buffer, and the keys it sees.
            auto q_row = [&](int i) -> const __nv_bfloat16* {
                const int tok = i / p.group, j = g * p.group + i - tok * p.group;
                return p.qkv + static_cast<long long>(q.row0 + tok0 + tok) * p.ld_qkv +
                       static_cast<long long>(j / p.heads_per_shard) * p.shard_w + (j % p.heads_per_shard) * D;
            };
            const bool upper = rows > 8;
            int lim[2];
            uint32_t qf[D / 16][4];
            float row_scale[2] = {p.scale_log2, p.scale_log2};
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int i = r0 + 8 * h;
                lim[h] = i < rows ? token_keys(q, keys, tok0 + i / p.group) : 0;
                const __nv_bfloat16* x = i < rows ? q_row(i) : nullptr;
                if constexpr (!E4M3) {
#pragma unroll
                    for (int ks = 0; ks < D / 16; ++ks) {
                        qf[ks][h] = x ? *reinterpret_cast<const uint32_t*>(x + ks * 16 + 2 * t) : 0u;
                        qf[ks][h + 2] = x ? *reinterpret_cast<const uint32_t*>(x + ks * 16 + 8 + 2 * t) : 0u;
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
                    row_scale[h] = p.scale_log2 * __int_as_float((127 - 14 + ex) << 23);
#pragma unroll
                    for (int hh = 0; hh < D / 64; ++hh)
#pragma unroll
                        for (int j = 0; j < 4; ++j)
#pragma unroll
                            for (int c = 0; c < 2; ++c) {
                                const float2 f = unpack_bf16x2(raw4[hh][j * 2 + c]);
                                qf[hh * 4 + j][h + 2 * c] = pack_f16x2(f.x * down, f.y * down);
                            }
                }
            }
            float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};
            float mv[2] = {-INFINITY, -INFINITY};  // 8-bit cache: reference of the weights 2^x vs
            float o[D / 8][4];
#pragma unroll
            for (int c = 0; c < D / 8; ++c)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[c][e] = 0.0f;

            for (int i = 0; i < seg; ++i, ++n) {
                if (C::WPB < NW && (n & 1) != warp / C::WPB) continue;
                const int st = n % NST;
                ok = ok && wait(full0 + 8 * st, (n / NST) & 1);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) continue;
                const uint32_t sk = base + st * C::STAGE, sv = sk + C::TILE;
                const int wk0 = wk * (16 * NG), key0 = (kb0 + i) * KB + wk0;  // the warp's keys of the block
                float s[NG][2][4] = {};
#pragma unroll
                for (int gr = 0; gr < NG; ++gr) {
                    if constexpr (!E4M3) {
                        // Matrices (keys 0-7, 8-15) x (d 0-7, 8-15) of a step: lanes 0-7 and 16-23 address keys
                        // 0-7 and 8-15 of the step's first eight d, lanes 8-15 and 24-31 of its second eight.
                        const uint32_t kr = wk0 + gr * 16 + (lane & 7) + ((lane >> 4) << 3), kc = (lane >> 3) & 1;
#pragma unroll
                        for (int ks = 0; ks < D / 16; ++ks) {
                            uint32_t b[4];
                            ldsm4(sk + (ks >> 2) * (KB * 128) + swz<128>(kr, (ks & 3) * 2 + kc), b);
                            mma<false>(s[gr][0], qf[ks], b[0], b[1]);
                            mma<false>(s[gr][1], qf[ks], b[2], b[3]);
                        }
                    } else {
#pragma unroll
                        for (int hh = 0; hh < D / 64; ++hh)
#pragma unroll
                            for (int nt = 0; nt < 2; ++nt) {
                                const uint4 u = ld_shared_v4(sk + swz<C::SEG>(wk0 + gr * 16 + nt * 8 + r0, hh * 4 + t));
                                const uint32_t c[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                                for (int j = 0; j < 4; ++j)
                                    mma<true>(s[gr][nt], qf[hh * 4 + j], e4m3x2_f16x2(c[j]), e4m3x2_f16x2(c[j] >> 16));
                            }
                    }
                }
                // Scores in the exp2 domain, masked; lane t has keys 2t, 2t + 1 of each eight.
                float lv[NG][2][2] = {};
#pragma unroll
                for (int gr = 0; gr < NG; ++gr)
#pragma unroll
                    for (int nt = 0; nt < 2; ++nt) {
                        float ks[2] = {1.0f, 1.0f};
                        if constexpr (E4M3) {
                            const float* sc = reinterpret_cast<const float*>(gbase + C::SC_OFF + st * C::SCALES) + wk0 +
                                              gr * 16 + nt * 8 + 2 * t;
                            const float2 k2 = *reinterpret_cast<const float2*>(sc);
                            const float2 v2 = *reinterpret_cast<const float2*>(sc + KB);
                            ks[0] = k2.x;
                            ks[1] = k2.y;
                            lv[gr][nt][0] = __log2f(v2.x);
                            lv[gr][nt][1] = __log2f(v2.y);
                        }
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int key = key0 + gr * 16 + nt * 8 + 2 * t + (e & 1);
                            const float x = s[gr][nt][e] * (ks[e & 1] * row_scale[e >> 1]);
                            s[gr][nt][e] = key < lim[e >> 1] ? x : -INFINITY;
                        }
                    }
                uint32_t pa[NG][4] = {};
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    if (h == 1 && !upper) break;  // no query in the tile's rows 8..15
                    constexpr int NX = 4 * NG;
                    float x[NX];
#pragma unroll
                    for (int e = 0; e < NX; ++e) x[e] = s[e >> 2][(e >> 1) & 1][2 * h + (e & 1)];
                    float mx = x[0];
#pragma unroll
                    for (int e = 1; e < NX; ++e) mx = fmaxf(mx, x[e]);
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
                    bool move = mx > m[h] + RESCALE;
                    float alpha = 1.0f;
                    if (move) {
                        alpha = ex2(m[h] - mx);
                        m[h] = mx;
                    }
                    const float ref = m[h] == -INFINITY ? 0.0f : m[h];
                    float pr[NX], sum = 0.0f;
#pragma unroll
                    for (int e = 0; e < NX; ++e) {
                        pr[e] = ex2(x[e] - ref);
                        sum += pr[e];
                    }
                    l[h] = l[h] * alpha + sum;
                    if constexpr (E4M3) {
                        // Weights 2^(x + log2 vs) against their own largest, which stands for 2^15: fp16's range
                        // whatever the scales.  A weight is rounded to 2^-11 of itself, or to 2^-25 where
                        // it is below fp16's normal range, 2^-40 of the largest.
                        float y[NX];
#pragma unroll
                        for (int e = 0; e < NX; ++e) y[e] = x[e] == -INFINITY ? -INFINITY : x[e] + lv[e >> 2][(e >> 1) & 1][e & 1];
                        float my = y[0];
#pragma unroll
                        for (int e = 1; e < NX; ++e) my = fmaxf(my, y[e]);
                        my = fmaxf(my, __shfl_xor_sync(0xffffffffu, my, 1));
                        my = fmaxf(my, __shfl_xor_sync(0xffffffffu, my, 2));
                        move = my > mv[h];
                        alpha = 1.0f;
                        if (move) {
                            alpha = ex2(mv[h] - my);
                            mv[h] = my;
                        }
                        const float rv = (mv[h] == -INFINITY ? 0.0f : mv[h]) - 15.0f;
#pragma unroll
                        for (int e = 0; e < NX; ++e) pr[e] = ex2(y[e] - rv);
                    }
                    if (__any_sync(0xffffffffu, move)) {
#pragma unroll
                        for (int c = 0; c < D / 8; ++c) {
                            o[c][2 * h] *= alpha;
                            o[c][2 * h + 1] *= alpha;
                        }
                    }
#pragma unroll
                    for (int gr = 0; gr < NG; ++gr) {
                        pa[gr][h] = E4M3 ? pack_f16x2(pr[4 * gr], pr[4 * gr + 1]) : pack_bf16x2(pr[4 * gr], pr[4 * gr + 1]);
                        pa[gr][h + 2] = E4M3 ? pack_f16x2(pr[4 * gr + 2], pr[4 * gr + 3]) : pack_bf16x2(pr[4 * gr + 2], pr[4 * gr + 3]);
                    }
                }
                // O += P V.  Rows of V past the sequence's keys are whatever the page holds: cleared, since
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
                    // Matrices (keys 0-7, 8-15) x two neighbouring eights of 16-bit columns.
                    const uint32_t vr = wk0 + gr * 16 + (lane & 15), vc = lane >> 4;
                    if constexpr (!E4M3) {
#pragma unroll
                        for (int c = 0; c < D / 16; ++c) {
                            uint32_t b[4];
                            ldsm4_t(sv + (c >> 2) * (KB * 128) + swz<128>(vr, (c & 3) * 2 + vc), b);
                            if (tail) {
                                b[0] &= live[0];
                                b[1] &= live[1];
                                b[2] &= live[0];
                                b[3] &= live[1];
                            }
                            mma<false>(o[2 * c], pa[gr], b[0], b[1]);
                            mma<false>(o[2 * c + 1], pa[gr], b[2], b[3]);
                        }
                    } else {
                        // A 16-bit column is two codes, d and d + 1: a register holds them for two keys.  Even and
                        // odd d go to two products: o[2 c'] has the even d of 16, o[2 c' + 1] the odd.
#pragma unroll
                        for (int c = 0; c < D / 32; ++c) {
                            uint32_t b[4];
                            ldsm4_t(sv + swz<C::SEG>(vr, c * 2 + vc), b);
                            if (tail) {
                                b[0] &= live[0];
                                b[1] &= live[1];
                                b[2] &= live[0];
                                b[3] &= live[1];
                            }
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                const uint32_t x = b[2 * h], y = b[2 * h + 1];
                                mma<true>(o[4 * c + 2 * h], pa[gr], e4m3x2_f16x2(__byte_perm(x, 0, 0x0020)),
                                          e4m3x2_f16x2(__byte_perm(y, 0, 0x0020)));
                                mma<true>(o[4 * c + 2 * h + 1], pa[gr], e4m3x2_f16x2(__byte_perm(x, 0, 0x0031)),
                                          e4m3x2_f16x2(__byte_perm(y, 0, 0x0031)));
                            }
                        }
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(empty0 + 8 * st);
            }

            // ---- merge the eight warps' sums over their keys
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
                l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
                if (t == 0) xm[warp * R + r0 + 8 * h] = m[h];
            }
            named_bar_sync(1, 32 * NW);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int i = r0 + 8 * h;
                float mm = -INFINITY;
#pragma unroll
                for (int x = 0; x < NW; ++x) mm = fmaxf(mm, xm[x * R + i]);
                // 2^(own reference - common one); the 8-bit cache's weights have a reference of their own.
                const float f = m[h] == -INFINITY ? 0.0f : ex2(m[h] - mm);
                float fo = f;
                if constexpr (E4M3) fo = mv[h] == -INFINITY ? 0.0f : ex2(mv[h] - 15.0f - mm);
                if (t == 0) xl[warp * R + i] = l[h] * f;
                if (i < rows) {
                    float* dst = acc_s + (warp * R + i) * C::LD_ACC;
                    if constexpr (!E4M3) {
#pragma unroll
                        for (int c = 0; c < D / 8; ++c)
                            *reinterpret_cast<float2*>(dst + c * 8 + 2 * t) =
                                make_float2(o[c][2 * h] * fo, o[c][2 * h + 1] * fo);
                    } else {
#pragma unroll
                        for (int c = 0; c < D / 16; ++c)
                            *reinterpret_cast<float4*>(dst + c * 16 + 4 * t) =
                                make_float4(o[2 * c][2 * h] * fo, o[2 * c + 1][2 * h] * fo, o[2 * c][2 * h + 1] * fo,
                                            o[2 * c + 1][2 * h + 1] * fo);
                    }
                }
            }
            named_bar_sync(1, 32 * NW);
            const bool begins = kb0 == 0, ends = kb0 + seg == w.nkb;
            const int slot = begins ? 1 : 0;
            if (ok) {
                for (int x = threadIdx.x; x < rows * (D / 4); x += 32 * NW) {
                    const int i = x / (D / 4), c = (x % (D / 4)) * 4;
                    float4 a = make_float4(0, 0, 0, 0);
                    float lt = 0.0f, mm = -INFINITY;
#pragma unroll
                    for (int y = 0; y < NW; ++y) {
                        const float4 b = *reinterpret_cast<const float4*>(acc_s + (y * R + i) * C::LD_ACC + c);
                        a.x += b.x;
                        a.y += b.y;
                        a.z += b.z;
                        a.w += b.w;
                        lt += xl[y * R + i];
                        mm = fmaxf(mm, xm[y * R + i]);
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
                        if (c == 0) *reinterpret_cast<float2*>(p.part_ml + at * 2) = make_float2(mm, lt);
                    }
                }
                if (begins && !ends && threadIdx.x == 0) {
                    // The tile's last block is in CTA (first block + blocks - 1) / per.
                    const long long at = share.begin + share.count - seg;
                    const int last = share_of(at + w.nkb - 1, share.per);
                    p.desc[blockIdx.x] = make_int4(q.row0 + tok0, g, rows, last - static_cast<int>(blockIdx.x) + 1);
                }
            }
        }
    }
    __syncthreads();
}

// Joins the parts of the tile that begins in slot 1 of CTA blockIdx.x and goes
// on in slot 0 of the next ones: O = sum 2^(m_i - m) O_i / sum 2^(m_i - m) l_i,
// in the order of the keys.  A warp takes 128 / D rows at a time, 16 bytes a
// lane.  zero_rest: also clears the rows of O that no sequence owns.
template <int D, int ROWS>
__global__ void __launch_bounds__(ROWS == R ? 256 : 1024) attn_join_kernel(PagedView v, int group, int heads, const float* part_o,
                                                                           const float* part_ml, const int4* desc,
                                                                           __nv_bfloat16* o, int zero_rest) {
    pdl_trigger();
    pdl_wait();
    constexpr int LANES = D / 4, PER_WARP = 32 / LANES;
    const int4 x = desc[blockIdx.x];  // the tile's first row, KV head, rows, parts
    if (zero_rest) {
        const int a = imin(imax(v.q_start[0], 0), v.rows), b = imin(imax(v.q_start[v.n_seqs], a), v.rows);
        const long long per = static_cast<long long>(heads) * D / 8;
        const long long threads = static_cast<long long>(gridDim.x) * blockDim.x;
        const long long me = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x;
        uint4* y = reinterpret_cast<uint4*>(o);
        for (long long i = me; i < a * per; i += threads) y[i] = make_uint4(0, 0, 0, 0);
        for (long long i = b * per + me; i < v.rows * per; i += threads) y[i] = make_uint4(0, 0, 0, 0);
    }
    const int c = (threadIdx.x % LANES) * 4;
    for (int i = threadIdx.x / LANES; i < x.z; i += (blockDim.x / 32) * PER_WARP) {
        if (x.w == 0) return;
        // Slot 1 of the first CTA is followed in memory by slot 0 of the next; then every second slot.
        auto slot = [&](int k) { return (static_cast<long long>(blockIdx.x) * 2 + (k == 0 ? 1 : 2 * k)) * ROWS + i; };
        float m = -INFINITY, l = 0.0f;
        float4 a = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
        for (int k = 0; k < x.w; ++k) {
            const float2 ml = *reinterpret_cast<const float2*>(part_ml + slot(k) * 2);
            const float4 b = *reinterpret_cast<const float4*>(part_o + slot(k) * D + c);
            const float mm = fmaxf(m, ml.x), base = mm == -INFINITY ? 0.0f : mm;
            const float f = ex2(m - base), e = ex2(ml.x - base);  // 2^-inf = 0: nothing before, nothing seen
            m = mm;
            l = l * f + ml.y * e;
            a.x = a.x * f + b.x * e;
            a.y = a.y * f + b.y * e;
            a.z = a.z * f + b.z * e;
            a.w = a.w * f + b.w * e;
        }
        const float inv = l != 0.0f ? 1.0f / l : 0.0f;
        const int tok = i / group;
        __nv_bfloat16* y = o + (static_cast<long long>(x.x + tok) * heads + x.y * group + i - tok * group) * D + c;
        *reinterpret_cast<uint2*>(y) = make_uint2(pack_bf16x2(a.x * inv, a.y * inv), pack_bf16x2(a.z * inv, a.w * inv));
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
    p.tile_tok = R / p.group;
    p.log2_tok = exact_log2(p.tile_tok);
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
                  tpi::launch_pdl(attn_few_kernel<C>, dim3(grid), dim3(NT), C::SMEM, stream, p), err);
    if (rc) return rc;
    return tpi::attn_join_launch(a, R, O, w, s, grid, zero_rest, stream, err);
}

template <int D, int ROWS>
cudaError_t join(const tpi::PagedArgs& a, void* O, uint8_t* w, const Scratch& s, int grid, bool zero_rest,
                 cudaStream_t stream) {
    return tpi::launch_pdl(attn_join_kernel<D, ROWS>, dim3(grid), dim3(ROWS == R ? 256 : 1024), 0, stream,
                           tpi::paged_view(a), a.heads / a.kv_heads, a.heads,
                           reinterpret_cast<const float*>(w + s.o), reinterpret_cast<const float*>(w + s.ml),
                           reinterpret_cast<const int4*>(w + s.desc), static_cast<__nv_bfloat16*>(O), zero_rest ? 1 : 0);
}

}  // namespace

namespace tpi {

// The kernel for many rows has the larger tiles.
size_t attn_paged_scratch_bytes(int head_dim) { return scratch_of(device_sm_count(), 128, head_dim).total; }

int attn_join_launch(const PagedArgs& a, int slot_rows, void* O, uint8_t* w, const Scratch& s, int grid,
                     bool zero_rest, cudaStream_t stream, std::string* err) {
    cudaError_t e;
    if (a.head_dim == 128)
        e = slot_rows == R ? join<128, R>(a, O, w, s, grid, zero_rest, stream)
                           : join<128, 128>(a, O, w, s, grid, zero_rest, stream);
    else
        e = slot_rows == R ? join<64, R>(a, O, w, s, grid, zero_rest, stream)
                           : join<64, 128>(a, O, w, s, grid, zero_rest, stream);
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
    // of 16.  More: tiles of 128 on tcgen05.
    const int group = a.heads / a.kv_heads;
    const int64_t most = a.max_new > 0 && a.max_new < a.tokens ? a.max_new : a.tokens;
    if (most * group > R)
        return attn_chunk_launch(a, O, scratch, zero_rest, stream, err);
    if (a.head_dim == 128)
        return a.e4m3 ? launch_few<Cfg<128, true, 4, 2, 4>>(a, O, scratch, zero_rest, stream, err)
                      : launch_few<Cfg<128, false, 4, 1, 4>>(a, O, scratch, zero_rest, stream, err);
    return a.e4m3 ? launch_few<Cfg<64, true, 4, 2, 6>>(a, O, scratch, zero_rest, stream, err)
                  : launch_few<Cfg<64, false, 4, 2, 4>>(a, O, scratch, zero_rest, stream, err);
}

}  // namespace tpi
