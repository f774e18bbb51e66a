// tp_verify.cu -- verification of drafted tokens against the target's
// probabilities, from given random numbers.
//
// With p = softmax(z / T) of the target and q = softmax(y / T) of the draft, a
// drafted x is taken when u q(x) < p(x), that is with probability
// min(1, p(x) / q(x)); where one is refused the next token is drawn from
// max(0, p - q) (normalised), so that the tokens follow p.  The draw is an
// exponential race: with E_v independent Exp(1), argmax_v w_v / E_v is v with
// probability w_v / sum w, whatever the scale of w, so that neither the sum
// nor a running sum over the vocabulary is needed.
//
// One launch: a cluster of 8 CTAs per sequence, an eighth of the vocabulary
// each.  Two rows at a time (up to four rows of logits with the draft's) are
// summed with a running maximum a thread; only the maxima and sums are
// exchanged, through distributed shared memory, as the vocabulary-parallel loss
// does between its shards, and every CTA decides by itself.  Rows behind a
// refused draft are not read, unless they are the other of its two.  The race
// then runs over the row where the drafts stop (its logits a second time, from
// L2).  A producer warp brings everything through a ring of bulk copies, 48 KB
// in flight a CTA, four CTAs an SM.  The floor is the logits' bytes; about five
// instructions a logit (unpacking, the maximum, a product, 2^x, a sum) come to
// half of that time, so the sums are kept short: the four states stay in
// registers and are joined across lanes once for both rows.  Measured: 64
// sequences of 2 to 5 drafts over 128256 words 48 us with fresh logits, 44.6 with
// the same ones again, where the rows that are needed take 24 at the memory's
// rate.  Neither memory (3.0 TB/s) nor issue (49% of the slots) is at its limit: a
// batch's decision waits for its last logits and an exchange of the cluster, and
// the producer with it, so that the ring is empty when the next batch begins.  2
// sequences of 3 drafts over 32768 words 11.3 us, all of it latency: a batch's
// loads, sums and exchange take about 2.5 us, the race as much.  Four rows a batch
// brought that to 10.3 but 64 sequences from 43.7 to 53 and a refused first draft
// from 4.4 to 6.2; deeper rings and prefetches of later rows changed nothing.
//
// A wait that gives up (2 s) tells every CTA of the cluster with its statistics,
// and the sequence's answer is -1 everywhere.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <string>

#include "tp_attn_paged.cuh"
#include "tp_device.cuh"
#include "tp_internal.h"
#include "tp_packed.cuh"

namespace {

using namespace tpk;

constexpr int CS = 8;      // CTAs of a cluster
constexpr int WARPS = 8;   // that sum; a ninth produces
constexpr int VT = WARPS * 32;
constexpr int ROWS = 2;    // rows of a batch
constexpr int ITEMS = 2 * ROWS;
constexpr int PPT = 4;     // pieces of 8 logits (16 bytes) of a thread in a stage of the ring
constexpr int NST = 3;     // stages of the ring
constexpr int TURN = PPT / 2 * VT;  // pieces of the race's turn: of both rows in a stage, their noise in the next
constexpr float LOG2E = 1.4426950408889634f;

struct VerifyParams {
    const __nv_bfloat16 *z, *y;
    long long rows, v;
    const int32_t *ids, *q_start;
    const float *temperature, *u, *noise;
    int32_t *accepted, *tokens;
    int give_up;  // self test: 1 or 2, the summing warps' waits give up at the first batch, or at the race
};

__device__ __forceinline__ float ex2f(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// m and s = sum 2^(x_v it - m), it = log2(e) / T, with m the largest x_v it of
// those summed so far as it is rounded: every use of m takes that same number,
// so its rounding cancels, as long as 2^(its rounding) is an ordinary number: the
// largest x_v it lies within 8 of an m below NEAR.  From there on the products are rounded
// like m, so that the largest stands for 1; other bf16 logits lie 2^19 below it or more.
// m = -inf: nothing yet.
struct Stat {
    float m, s;
};
constexpr float NEAR = 268435456.0f;  // 2^28
// 1 / T as logits are scaled by it, and the |m| below which they are scaled and subtracted in one step: none for an
// infinite T, where that step would take -inf times 0.
struct Scale {
    float it, near;
};
// x it, held to the finite numbers: a logit at the type's ends stays one, only
// -inf is no probability.
__device__ __forceinline__ float scaled(float x, float it) {
    return x == -INFINITY ? x : fminf(fmaxf(x * it, -3.4028234663852886e38f), 3.4028234663852886e38f);
}
// 2^(x it - m).  The product is not rounded by itself below `near`.
__device__ __forceinline__ float weight(float x, Scale t, float m) {
    return fabsf(m) < t.near ? ex2f(fmaf(x, t.it, -m)) : ex2f(scaled(x, t.it) - m);
}

// Largest value and its lowest index.
struct Best {
    float v;
    int i;
};
__device__ __forceinline__ Best better(Best a, Best b) {
    return (b.v > a.v || (b.v == a.v && b.i < a.i)) ? b : a;
}
__device__ __forceinline__ Best warp_best(Best a) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const Best b = {__shfl_xor_sync(0xffffffffu, a.v, o), __shfl_xor_sync(0xffffffffu, a.i, o)};
        a = better(a, b);
    }
    return a;
}
// Joins the states of lanes that differ in the low bits of `span` (8 or 32 lanes): one maximum, then one sum.
template <int SPAN>
__device__ __forceinline__ Stat join_lanes(Stat a) {
    float m = a.m;
#pragma unroll
    for (int o = SPAN / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    float s = a.m == -INFINITY ? 0.0f : a.s * ex2f(a.m - m);
#pragma unroll
    for (int o = SPAN / 2; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    return {m, s};
}
// As join_lanes, of largest logits (m the value, s the index's bits).
template <int SPAN>
__device__ __forceinline__ Stat best_lanes(Stat a) {
    Best c = {a.m, __float_as_int(a.s)};
#pragma unroll
    for (int o = SPAN / 2; o > 0; o >>= 1)
        c = better(c, {__shfl_xor_sync(0xffffffffu, c.v, o), __shfl_xor_sync(0xffffffffu, c.i, o)});
    return {c.v, __int_as_float(c.i)};
}

// 8 bytes to the same shared-memory address in CTA `rank` of the cluster.
__device__ __forceinline__ void store_cluster(uint32_t addr, int rank, uint32_t a, uint32_t b) {
    asm volatile("st.shared::cluster.v2.b32 [%0], {%1, %2};" ::"r"(mapa_shared(addr, static_cast<uint32_t>(rank))), "r"(a),
                 "r"(b)
                 : "memory");
}

__device__ __forceinline__ float prob(float x, Scale t, Stat st) {
    return st.s > 0.0f ? weight(x, t, st.m) / st.s : 0.0f;
}

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// What few calls need stays out of line, and a batch's rows share one loop's code: less to fetch in a call that
// runs it once (97 -> 64 KB; 2 sequences of 3 drafts 11.7 -> 11.3 us, 64 sequences as before).

// sum_pieces from `near` on: low temperatures, an infinite one, logits at the type's ends.  m: the new maximum.
__device__ __noinline__ Stat sum_ends(Stat a, uint4 u1, uint4 u2, float it, float m) {
    const uint32_t w[8] = {u1.x, u1.y, u1.z, u1.w, u2.x, u2.y, u2.z, u2.w};
    float sum = 0.0f;
#pragma unroll
    for (int k = 0; k < 8; ++k) sum += ex2f(scaled(bf16_lo(w[k]), it) - m) + ex2f(scaled(bf16_hi(w[k]), it) - m);
    return {m, fmaf(a.s, ex2f(a.m - m), sum)};
}

// Two pieces of logits into a running state (u2 only if both).
__device__ __forceinline__ void sum_pieces(Stat& a, const uint4& u1, const uint4& u2, Scale t) {
    const float it = t.it;
    const uint32_t w[8] = {u1.x, u1.y, u1.z, u1.w, u2.x, u2.y, u2.z, u2.w};
    float v[16];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        v[2 * k] = bf16_lo(w[k]);
        v[2 * k + 1] = bf16_hi(w[k]);
    }
    float bm[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) bm[k] = max3(fmaxf(v[k], v[k + 4]), v[k + 8], v[k + 12]);
    const float m = fmaxf(a.m, scaled(max3(fmaxf(bm[0], bm[1]), bm[2], bm[3]), it));
    if (!(fabsf(m) < t.near)) {  // nothing but -inf so far, or from `near` on
        if (m != -INFINITY) a = sum_ends(a, u1, u2, it, m);
        return;
    }
    float x[16];
    const uint64_t its = f2_pack(it, it), minus = f2_pack(-m, -m);
#pragma unroll
    for (int k = 0; k < 8; ++k) f2_unpack(f2_fma(f2_pack(v[2 * k], v[2 * k + 1]), its, minus), x[2 * k], x[2 * k + 1]);
    uint64_t sum[4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
        sum[k] = f2_add(f2_pack(ex2f(x[4 * k]), ex2f(x[4 * k + 1])), f2_pack(ex2f(x[4 * k + 2]), ex2f(x[4 * k + 3])));
    float lo, hi;
    f2_unpack(f2_add(f2_add(sum[0], sum[1]), f2_add(sum[2], sum[3])), lo, hi);
    a.s = fmaf(a.s, ex2f(a.m - m), lo + hi);
    a.m = m;
}

// The first of the largest logits: m the value, s the index's bits.
__device__ __noinline__ Stat best_piece(Stat a, uint4 u, int index) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        const float v = (k & 1) ? bf16_hi(w[k >> 1]) : bf16_lo(w[k >> 1]);
        if (v > a.m) a = {v, __int_as_float(index + k)};  // indices ascend in a thread
    }
    return a;
}
// Two logits' weights.
__device__ __forceinline__ uint64_t weight2(uint32_t w, uint64_t its, uint64_t minus) {
    float x0, x1;
    f2_unpack(f2_fma(f2_pack(bf16_lo(w), bf16_hi(w)), its, minus), x0, x1);
    return f2_pack(ex2f(x0), ex2f(x1));
}

// The same two of p - r q from `near` on.
__device__ __noinline__ uint64_t weight2_ends(uint32_t z, uint32_t y, Scale t, float zm, float ym, float r) {
    float a0 = weight(bf16_lo(z), t, zm), a1 = weight(bf16_hi(z), t, zm);
    if (r != 0.0f) {
        a0 = fmaf(-r, weight(bf16_lo(y), t, ym), a0);
        a1 = fmaf(-r, weight(bf16_hi(y), t, ym), a1);
    }
    return f2_pack(a0, a1);
}

__global__ void __cluster_dims__(CS, 1, 1) __launch_bounds__(VT + 32, 4) verify_kernel(const VerifyParams p) {
    extern __shared__ uint4 ring_raw[];
    uint4(*ring)[PPT * VT] = reinterpret_cast<uint4(*)[PPT * VT]>(ring_raw);  // [NST]
    __shared__ alignas(8) uint64_t bars[2 * NST];  // full, empty
    __shared__ Stat part[ITEMS][WARPS];            // by row of logits: a warp's statistics, or its largest logit
    __shared__ Stat all[2][ITEMS][CS];             // by batch parity, row of logits and CTA
    __shared__ Best race[WARPS], raced[2][CS];     // of a warp; by attempt and CTA
    // Of 64 rows: the drafted token (-1: none, or outside), its logits, and the random number.  Halves of 32 rows
    // are filled in turn: the half written is two batches at least from any that is read.
    __shared__ int xs[64];
    __shared__ float zs[64], ys[64], us[64];
    __shared__ int abort_word;
    const int rank = static_cast<int>(cluster_ctarank()), warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int tid = static_cast<int>(threadIdx.x), s = blockIdx.x / CS;
    const uint32_t full0 = smem_u32(bars), empty0 = full0 + 8 * NST;
    if (tid == 0) {
        for (int i = 0; i < NST; ++i) {
            mbar_init(full0 + 8 * i, 1);
            mbar_init(empty0 + 8 * i, WARPS);
        }
        abort_word = 0;
        fence_barrier_init();
    }
    // Every CTA of the cluster runs, and its barriers are there, before one stores into another's shared memory.
    __syncwarp();
    cluster_arrive();
    pdl_trigger();
    pdl_wait();
    cluster_wait();
    const long long r0 = min(max(static_cast<long long>(p.q_start[s]), 0ll), p.rows);
    const long long r1 = min(max(static_cast<long long>(p.q_start[s + 1]), r0), p.rows);
    const float T = p.temperature ? p.temperature[s] : 1.0f;
    const int n = static_cast<int>(r1 - r0);
    if (n == 0) {  // the whole cluster
        if (rank == 0 && tid == 0) p.accepted[s] = 0;
        return;
    }
    const bool greedy = !(T > 0.0f);
    const float it = fminf(LOG2E / T, 1e30f);
    const Scale scale = {it, it > 0.0f ? NEAR : 0.0f};
    const int pieces = static_cast<int>(p.v / 8), mine = (pieces + CS - 1) / CS;
    const int begin = min(rank * mine, pieces), end = min(begin + mine, pieces);

    const Waiter wait = {&abort_word, nullptr, 2000000000ull};
    bool ok = true;
    // Self test: from here on no wait of the summing warps succeeds, while copies are on their way.
    auto give_up = [&](int where) {
        if (p.give_up == where && warp < WARPS) {
            *reinterpret_cast<volatile int*>(&abort_word) = 1;
            ok = false;
        }
    };
    give_up(1);
    // Ring position, the same sequence in the producer and in those that sum.
    int st = 0, issued = 0;
    uint32_t phase = 0;
    auto advance = [&] {
        if (++st == NST) {
            st = 0;
            phase ^= 1;
        }
    };
    // Producer: the next stage gets `bytes` from a at offset 0, and more from b at the stage's middle.
    auto produce = [&](const void* a, uint32_t bytes, const void* b, uint32_t more) {
        // Warps that gave up release their stages unread: a barrier whose copy has not arrived must not be armed again.
        ok = ok && wait(empty0 + 8 * st, phase ^ 1) && !*reinterpret_cast<volatile int*>(&abort_word);
        if (!ok) return;
        const uint32_t full = full0 + 8 * st;
        mbar_arrive_expect_tx(full, bytes + more);
        if (bytes) bulk_load(smem_u32(&ring[st][0]), a, bytes, full);
        if (more) bulk_load(smem_u32(&ring[st][TURN]), b, more, full);
        ++issued;
        advance();
    };
    auto release = [&] {
        __syncwarp();
        if (lane == 0) mbar_arrive(empty0 + 8 * st);
        advance();
    };
    // The noise of this CTA's words comes to L2 meanwhile.
    if (!greedy && p.noise && tid == VT && end > begin)
        asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(p.noise + s * p.v + begin * 8),
                     "r"(static_cast<uint32_t>(end - begin) * 32u)
                     : "memory");

    int taken = n - 1, token = -1;
    Stat sp = {-INFINITY, 0.0f}, sq = {-INFINITY, 0.0f};
    bool drafted = false;  // the row that stops has a draft distribution
    bool failed = false;   // a wait of some CTA gave up: what was summed is not the rows' sums, and nothing is settled
    for (int b0 = 0, parity = 0; b0 < n; b0 += ROWS, parity ^= 1) {
        const int rows = min(ROWS, n - b0);
        // Rows of logits: the target's, then the draft's (none behind the last draft).
        const int drafts = greedy || !p.y ? 0 : min(rows, n - 1 - b0), items = rows + drafts;
        auto row_of = [&](int i) {
            return reinterpret_cast<const uint4*>(i < rows ? p.z + (r0 + b0 + i) * p.v : p.y + (r0 + b0 + i - rows) * p.v);
        };
        if (warp == WARPS) {
            if (lane == 0)
                for (int i = 0; i < items; ++i)
                    for (int at = begin; at < end; at += PPT * VT)
                        produce(row_of(i) + at, static_cast<uint32_t>(min(PPT * VT, end - at)) * 16u, nullptr, 0);
            __syncwarp();
            if (b0 % 32 == 0) {  // what the decisions of 32 rows read, while the logits are summed
                const long long r = r0 + b0 + lane;
                int x = -1;
                float zx = 0.0f, yx = 0.0f, ux = 0.0f;
                if (b0 + lane + 1 < n) {
                    x = p.ids[r + 1];
                    ux = p.u[r];
                    if (x >= p.v) x = -1;
                    if (x >= 0) {
                        zx = __bfloat162float(p.z[r * p.v + x]);
                        if (!greedy && p.y) yx = __bfloat162float(p.y[r * p.v + x]);
                    }
                }
                const int at = (b0 + lane) % 64;
                xs[at] = x < 0 ? -1 : x;
                zs[at] = zx;
                ys[at] = yx;
                us[at] = ux;
            }
        } else {
            Stat a[ITEMS];
#pragma unroll
            for (int i = 0; i < ITEMS; ++i) a[i] = {-INFINITY, 0.0f};
#pragma unroll 1
            for (int i = 0; i < items; ++i) {
                Stat b = {-INFINITY, 0.0f};
                for (int at = begin; at < end; at += PPT * VT) {
                    ok = ok && wait(full0 + 8 * st, phase);
                    if (ok) {
                        const uint4 none = make_uint4(0xff80ff80u, 0xff80ff80u, 0xff80ff80u, 0xff80ff80u);  // bf16 -inf
#pragma unroll
                        for (int e = 0; e < PPT; e += 2) {  // this thread's pieces: at + e VT + tid
                            const int left = end - at - e * VT - tid;
                            if (left <= 0) break;
                            const uint4 u1 = ring[st][e * VT + tid], u2 = left > VT ? ring[st][(e + 1) * VT + tid] : none;
                            if (greedy) {
                                b = best_piece(b, u1, (at + e * VT + tid) * 8);
                                b = best_piece(b, u2, (at + (e + 1) * VT + tid) * 8);
                            } else {
                                sum_pieces(b, u1, u2, scale);
                            }
                        }
                    }
                    release();
                }
#pragma unroll
                for (int k = 0; k < ITEMS; ++k)
                    if (k == i) a[k] = b;
            }
#pragma unroll
            for (int i = 0; i < ITEMS; ++i) a[i] = greedy ? best_lanes<32>(a[i]) : join_lanes<32>(a[i]);
            if (lane == 0)
#pragma unroll
                for (int i = 0; i < ITEMS; ++i) part[i][warp] = a[i];
        }
        __syncthreads();
        // The CTA's statistics of each row, to every CTA of the cluster.
        static_assert(ITEMS * WARPS == 32 && ITEMS * CS == 32, "a lane a row and warp, or a row and CTA");
        if (warp == 0) {
            Stat b = part[lane / WARPS][lane % WARPS];
            b = greedy ? best_lanes<WARPS>(b) : join_lanes<WARPS>(b);  // in every lane of the row: one a CTA to tell
            if (abort_word) b.m = NAN;  // no largest value is NaN: a wait of this CTA gave up
            store_cluster(smem_u32(&all[parity][lane / CS][rank]), lane % CS, __float_as_uint(b.m), __float_as_uint(b.s));
        }
        // A batch's buffer is written again two batches on: behind the next batch's barrier, which every CTA
        // reaches after it has read this one.
        cluster_sync_all();
        // Every warp decides: the rows' statistics, 8 lanes each, then lane i row i.
        Stat b = all[parity][lane / CS][lane % CS];
        failed = __any_sync(0xffffffffu, isnan(b.m));  // the same in every warp and CTA
        if (failed) break;
        b = greedy ? best_lanes<CS>(b) : join_lanes<CS>(b);
        const int of_p = min(lane, rows - 1) * CS, of_q = min(rows + lane, ITEMS - 1) * CS;
        const Stat tp_ = {__shfl_sync(0xffffffffu, b.m, of_p), __shfl_sync(0xffffffffu, b.s, of_p)};
        Stat tq = {__shfl_sync(0xffffffffu, b.m, of_q), __shfl_sync(0xffffffffu, b.s, of_q)};
        if (lane >= drafts) tq = {-INFINITY, 0.0f};
        bool take = false;
        if (lane < rows) {
            const int at = (b0 + lane) % 64, x = xs[at];
            if (greedy) take = x >= 0 && tp_.m > -INFINITY && __float_as_int(tp_.s) == x;
            else if (x >= 0) take = us[at] * prob(ys[at], scale, tq) < prob(zs[at], scale, tp_);
        }
        const unsigned kept = __ballot_sync(0xffffffffu, lane < rows && !take);
        if (kept) {
            const int i = __ffs(kept) - 1;
            taken = b0 + i;
            sp = {__shfl_sync(0xffffffffu, tp_.m, i), __shfl_sync(0xffffffffu, tp_.s, i)};
            sq = {__shfl_sync(0xffffffffu, tq.m, i), __shfl_sync(0xffffffffu, tq.s, i)};
            drafted = i < drafts;
            break;
        }
    }
    if (greedy) {
        token = sp.m > -INFINITY ? __float_as_int(sp.s) : -1;
    } else if (!failed) {
        // The race over w = max(0, p - q); where that leaves nothing, a second one over p.
        give_up(2);
        const uint4* z = reinterpret_cast<const uint4*>(p.z + (r0 + taken) * p.v);
        const uint4* y = drafted && sq.s > 0.0f ? reinterpret_cast<const uint4*>(p.y + (r0 + taken) * p.v) : nullptr;
        const float4* noise = p.noise ? reinterpret_cast<const float4*>(p.noise + s * p.v) : nullptr;
        // p - q up to the factor 1 / p's sum.
        const float r = y ? sp.s / sq.s : 0.0f;
        const bool plain = fabsf(sp.m) < scale.near && (!y || fabsf(sq.m) < scale.near);
        for (int attempt = 0; attempt < 2; ++attempt) {
            if (warp == WARPS) {
                if (lane == 0)
                    for (int at = begin; at < end; at += TURN) {
                        const uint32_t m = static_cast<uint32_t>(min(TURN, end - at));
                        produce(z + at, m * 16, y ? y + at : nullptr, y ? m * 16 : 0);
                        produce(noise ? noise + 2 * at : nullptr, noise ? m * 32 : 0, nullptr, 0);
                    }
                __syncwarp();
            } else {
                // b.v is the best quotient so far: a word passes it if w - b.v e > 0, which few do.
                Best b = {0.0f, 0x7fffffff};
                const uint64_t its = f2_pack(it, it), zm = f2_pack(-sp.m, -sp.m), ym = f2_pack(-sq.m, -sq.m), minus_r = f2_pack(-r, -r);
                for (int at = begin; at < end; at += TURN) {
                    uint64_t w[TURN / VT][4];
                    ok = ok && wait(full0 + 8 * st, phase);
#pragma unroll
                    for (int h = 0; h < TURN / VT; ++h) {
                        if (!ok || at + h * VT + tid >= end) continue;
                        const uint4 u = ring[st][h * VT + tid], t = y ? ring[st][TURN + h * VT + tid] : make_uint4(0, 0, 0, 0);
                        const uint32_t zw[4] = {u.x, u.y, u.z, u.w}, yw[4] = {t.x, t.y, t.z, t.w};
                        if (plain) {
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                w[h][k] = weight2(zw[k], its, zm);
                                if (y) w[h][k] = f2_fma(minus_r, weight2(yw[k], its, ym), w[h][k]);
                            }
                        } else {
#pragma unroll
                            for (int k = 0; k < 4; ++k) w[h][k] = weight2_ends(zw[k], yw[k], scale, sp.m, sq.m, y ? r : 0.0f);
                        }
                    }
                    release();
                    ok = ok && wait(full0 + 8 * st, phase);
#pragma unroll
                    for (int h = 0; h < TURN / VT; ++h) {
                        if (!ok || at + h * VT + tid >= end) continue;
                        float4 ea = make_float4(1.0f, 1.0f, 1.0f, 1.0f), eb = ea;
                        if (noise) {
                            ea = reinterpret_cast<const float4*>(&ring[st][0])[2 * (h * VT + tid)];
                            eb = reinterpret_cast<const float4*>(&ring[st][0])[2 * (h * VT + tid) + 1];
                        }
                        const uint64_t e[4] = {f2_pack(ea.x, ea.y), f2_pack(ea.z, ea.w), f2_pack(eb.x, eb.y), f2_pack(eb.z, eb.w)};
                        const uint64_t minus_b = f2_pack(-b.v, -b.v);
                        float d[8];
#pragma unroll
                        for (int k = 0; k < 4; ++k) f2_unpack(f2_fma(minus_b, e[k], w[h][k]), d[2 * k], d[2 * k + 1]);
                        if (max3(max3(d[0], d[1], d[2]), max3(d[3], d[4], d[5]), fmaxf(d[6], d[7])) > 0.0f) {  // NaN is ignored
#pragma unroll
                            for (int k = 0; k < 8; ++k) {
                                float w0, w1, e0, e1;
                                f2_unpack(w[h][k >> 1], w0, w1);
                                f2_unpack(e[k >> 1], e0, e1);
                                const float wk = (k & 1) ? w1 : w0, q = __fdividef(wk, (k & 1) ? e1 : e0);
                                if (wk > 0.0f && q > b.v) b = {q, (at + h * VT + tid) * 8 + k};
                            }
                        }
                    }
                    release();
                }
                b = warp_best(b);
                if (lane == 0) race[warp] = b;
            }
            __syncthreads();
            if (tid < CS) {
                Best b = race[0];
#pragma unroll
                for (int k = 1; k < WARPS; ++k) b = better(b, race[k]);
                if (abort_word) b.v = NAN;
                store_cluster(smem_u32(&raced[attempt][rank]), tid, __float_as_uint(b.v), static_cast<uint32_t>(b.i));
            }
            __syncwarp();
            cluster_sync_all();
            Best b = raced[attempt][0];
            failed = isnan(b.v);
#pragma unroll
            for (int k = 1; k < CS; ++k) {
                failed = failed || isnan(raced[attempt][k].v);
                b = better(b, raced[attempt][k]);
            }
            if (failed) break;
            token = b.v > 0.0f && sp.s > 0.0f ? b.i : -1;
            if (token >= 0 || !y) break;  // the same in every CTA
            y = nullptr;
        }
    }
    // No copy may be in flight when the CTA's shared memory goes, whichever warp gave up.
    if (abort_word && tid == VT)
        for (int i = max(0, issued - NST); i < issued; ++i) drain(full0 + 8 * (i % NST), (i / NST) & 1);
    if (failed) taken = token = -1;
    if (rank == 0) {
        if (tid == 0) p.accepted[s] = taken;
        for (int i = tid; i < n; i += VT + 32)
            p.tokens[r0 + i] = i < taken ? p.ids[r0 + i + 1] : i == taken ? token : -1;
    }
}

}  // namespace

namespace tpi {

int verify_launch(const VerifyArgs& a, cudaStream_t stream, std::string* err) {
    if (a.n_seqs == 0) return TP_OK;
    VerifyParams p{};
    p.z = static_cast<const __nv_bfloat16*>(a.logits);
    p.y = static_cast<const __nv_bfloat16*>(a.draft_logits);
    p.rows = a.M;
    p.v = a.v;
    p.ids = a.ids;
    p.q_start = a.q_start;
    p.temperature = a.temperature;
    p.u = a.u;
    p.noise = a.noise;
    p.accepted = a.accepted;
    p.tokens = a.tokens;
    p.give_up = a.give_up;
    constexpr int SMEM = NST * PPT * VT * 16;
    static bool configured[64] = {false};
    int dev = 0;
    cudaGetDevice(&dev);
    cudaError_t e = cudaSuccess;
    if (dev < 64 && !configured[dev]) {
        e = cudaFuncSetAttribute(verify_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM);
        configured[dev] = e == cudaSuccess;
    }
    if (e == cudaSuccess)
        e = launch_pdl(verify_kernel, dim3(static_cast<unsigned>(a.n_seqs) * CS), dim3(VT + 32), SMEM, stream, p);
    if (e == cudaSuccess) e = cudaGetLastError();
    if (e != cudaSuccess) {
        if (err) *err = std::string("verification kernel: ") + cudaGetErrorString(e);
        return TP_ERR_CUDA;
    }
    return TP_OK;
}

}  // namespace tpi
