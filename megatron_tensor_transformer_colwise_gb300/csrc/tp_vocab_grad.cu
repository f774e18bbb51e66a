// tp_vocab_grad.cu -- the vocabulary's two ends in training: the scaled
// embedding lookup, the embedding's gradient, and the loss with the gradient of
// its logits.
//
// Source: "텐서 병렬화" (itwiki, Tensor parallelism), section "임베딩과
// 출력층" (embedding and output layer): the embedding matrix is split along
// the vocabulary, so shard i's gradient is rows [i v/t, (i+1) v/t) of dE, and
// the cross-entropy exchanges per-token statistics alone.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <string>

#include "tp_device.cuh"
#include "tp_internal.h"
#include "tp_packed.cuh"

namespace {

using namespace tpk;

constexpr float LOG2E = 1.4426950408889634f;

__device__ __forceinline__ float ex2f(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ void unpack8(const uint4& u, float (&f)[8]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const float2 p = unpack_bf16x2(w[e]);
        f[2 * e] = p.x;
        f[2 * e + 1] = p.y;
    }
}

__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
    return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
}

// ------------------------------------------------------------ scaled lookup

// One warp per token: out = scale * E[id] (rounded once), or zeros.  Eight
// 16-byte pieces a lane are read before the first is used: with one at a time the
// lanes waited for memory (8192 x 4096: 19.7 us).
constexpr int EMB_WARPS = 4, EMB_LOADS = 8;

__global__ void __launch_bounds__(EMB_WARPS * 32) embedding_scaled_kernel(const int32_t* ids, long long M,
                                                                         const __nv_bfloat16* E, long long v,
                                                                         int h, float scale, __nv_bfloat16* out) {
    pdl_trigger();
    pdl_wait();
    const long long m = static_cast<long long>(blockIdx.x) * EMB_WARPS + (threadIdx.x >> 5);
    if (m >= M) return;
    const long long id = ids[m];
    const bool owned = id >= 0 && id < v;
    const uint4* src = reinterpret_cast<const uint4*>(E + (owned ? id : 0) * h);
    uint4* dst = reinterpret_cast<uint4*>(out + m * h);
    const int nv = owned ? h >> 3 : 0;
    for (int c = threadIdx.x & 31; c < (h >> 3); c += 32 * EMB_LOADS) {
        uint4 u[EMB_LOADS];
#pragma unroll
        for (int k = 0; k < EMB_LOADS; ++k) u[k] = c + 32 * k < nv ? src[c + 32 * k] : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int k = 0; k < EMB_LOADS; ++k) {
            float f[8];
            unpack8(u[k], f);
#pragma unroll
            for (int e = 0; e < 8; ++e) f[e] = owned ? f[e] * scale : 0.0f;
            if (c + 32 * k < (h >> 3)) dst[c + 32 * k] = pack8(f);
        }
    }
}

// ------------------------------------------------------------ embedding gradient

// Two launches, the same bits every time:
//  1. tokens sorted by word;
//  2. the sorted tokens in parts of equal length, summed by word, and behind
//     these CTAs others that write the zeros of words without a token.  A word that
//     a part's border cuts leaves partial sums, and the last of its parts to
//     arrive (a counter that the first launch cleared) adds them in order.
// Parts of equal length keep a frequent word (in text, one token in ten is the
// same one) from being one CTA's work.
// Bound by the zeros' way to memory: 8192 tokens of 4096 over 128256 words 308 us
// (2.1 GB of dE; 320 us at the rate of a copy), 2048 of 1024 over 32768 29 us (20.4),
// of which the sorting launch is about 5 and a frequent word's last parts the end.
// Added to dE instead: 65 us (28) and 15.  With one CTA a word the first took 1100
// us, with the partial sums added by a third launch the second 42, with the zeros
// written by the sorting kernel 40.

// Sorting: a CTA owns BINS words and looks through all ids: it counts the
// tokens of words below its own (its place in the order) and of each of its
// own, then puts the positions down word by word.  Every warp takes a
// contiguous part of the tokens and has counters of its own, so the positions
// of a word come out ascending whatever the order of the work.
//   sorted: tokens by word; start[r] .. start[r + 1]: those of word r.
// As many warps (4 to 32) as have a batch of loads each: what a CTA does for its
// counters grows with them (64 tokens over 128256 words: 14.9 us with 32).
constexpr int BINS = 128, SORT_LOADS = 8, MAX_SORT_WARPS = 32;

struct Entry {
    int32_t word, at;  // a token's word and its position
};

// Calls f(id, position) for this lane's tokens of [from, to), 32 consecutive
// ones a warp and call; -1 past the end.
template <typename F>
__device__ __forceinline__ void for_ids(const int32_t* ids, long long from, long long to, F&& f) {
    const int lane = threadIdx.x & 31;
    for (long long at = from; at < to; at += 32 * SORT_LOADS) {
        int32_t id[SORT_LOADS];
#pragma unroll
        for (int k = 0; k < SORT_LOADS; ++k) {
            const long long i = at + 32 * k + lane;
            id[k] = i < to ? ids[i] : -1;
        }
#pragma unroll
        for (int k = 0; k < SORT_LOADS; ++k)
            if (at + 32 * k < to) f(id[k], at + 32 * k + lane);
    }
}

__global__ void __launch_bounds__(MAX_SORT_WARPS * 32) sort_tokens_kernel(const int32_t* ids, long long M, int v,
                                                                     Entry* sorted, int32_t* start,
                                                                     int32_t* counters, long long n_counters) {
    extern __shared__ int32_t counts[];  // [warps][BINS]
    int32_t(*count)[BINS] = reinterpret_cast<int32_t(*)[BINS]>(counts);
    __shared__ int32_t below[MAX_SORT_WARPS], sums[BINS / 32];
    const int warps = blockDim.x >> 5;
    pdl_trigger();
    pdl_wait();
    const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int lo = blockIdx.x * BINS, bins = min(BINS, v - lo);
    for (long long i = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x; i < n_counters;
         i += static_cast<long long>(gridDim.x) * blockDim.x)
        counters[i] = 0;
    for (int b = lane; b < BINS; b += 32) count[w][b] = 0;
    __syncwarp();
    const long long part = ((M + warps - 1) / warps + 31) / 32 * 32;
    const long long from = w * part, to = min(from + part, M);
    int under = 0;
    for_ids(ids, from, to, [&](int id, long long) {
        under += id >= 0 && id < lo;
        if (id >= lo && id - lo < bins) atomicAdd(&count[w][id - lo], 1);
    });
    under = __reduce_add_sync(0xffffffffu, under);
    if (lane == 0) below[w] = under;
    __syncthreads();
    // count[w][b] becomes the place of warp w's first token of word lo + b.
    int total = 0, base = 0;
    if (threadIdx.x < BINS) {
        for (int k = 0; k < warps; ++k) {
            const int n = count[k][threadIdx.x];
            count[k][threadIdx.x] = total;
            total += n;
            base += below[k];
        }
        int upto = total;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int n = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o) upto += n;
        }
        if (lane == 31) sums[w] = upto;
        base += upto - total;
    }
    __syncthreads();
    if (threadIdx.x < BINS) {
        for (int k = 0; k < w; ++k) base += sums[k];
        for (int k = 0; k < warps; ++k) count[k][threadIdx.x] += base;
        if (threadIdx.x < bins) start[lo + threadIdx.x] = base;
        if (lo + static_cast<int>(threadIdx.x) == v - 1) start[v] = base + total;
    }
    __syncthreads();
    for_ids(ids, from, to, [&](int id, long long i) {
        const bool mine = id >= lo && id - lo < bins;
        const unsigned live = __ballot_sync(0xffffffffu, mine);
        if (mine) {
            const int b = id - lo;
            const unsigned same = __match_any_sync(live, b);
            const unsigned before = same & ((1u << lane) - 1u);
            sorted[count[w][b] + __popc(before)] = {id, static_cast<int32_t>(i)};
            __syncwarp(live);
            if (!before) count[w][b] += __popc(same);
        }
        __syncwarp();
    });
}

// Columns (in eights) and sorted tokens of a CTA.
constexpr int SUM_THREADS = 128, MAX_PART = 512, SUM_LOADS = 8;

__device__ __forceinline__ void store_sum(float* row, int c, const float (&s)[8], float scale, int accumulate) {
    float4* out = reinterpret_cast<float4*>(row) + 2 * c;
    float4 a = make_float4(0.0f, 0.0f, 0.0f, 0.0f), b = a;
    if (accumulate) {
        a = out[0];
        b = out[1];
    }
    out[0] = make_float4(fmaf(scale, s[0], a.x), fmaf(scale, s[1], a.y), fmaf(scale, s[2], a.z), fmaf(scale, s[3], a.w));
    out[1] = make_float4(fmaf(scale, s[4], b.x), fmaf(scale, s[5], b.y), fmaf(scale, s[6], b.z), fmaf(scale, s[7], b.w));
}

// Zeros for the words without a token among `words` from `first` on, which are
// few enough for `from` to hold where their tokens start.
constexpr int CLEAR_BYTES = 65536, MAX_CLEAR = MAX_PART;  // of a CTA: bytes about, words at most

__device__ __forceinline__ void clear_words(const int32_t* start, long long first, int words, int h,
                                            float* dE, int32_t* from) {
    for (int k = threadIdx.x; k <= words; k += blockDim.x) from[k] = start[first + k];
    __syncthreads();
    // Short rows side by side, long ones by all threads.
    const int pieces = h >> 2, rows = max(1, static_cast<int>(blockDim.x) / pieces), mine = threadIdx.x / pieces;
    for (int r = rows > 1 ? mine : 0; mine < rows && r < words; r += rows) {
        if (from[r] != from[r + 1]) continue;
        float4* row = reinterpret_cast<float4*>(dE + (first + r) * h);
        for (int c = threadIdx.x - (rows > 1 ? mine * pieces : 0); c < pieces; c += blockDim.x)
            row[c] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    }
}

// CTAs [0, n_parts slices): sorted tokens [a part, (a + 1) part) for one slice of
// columns each; those behind them: zeros for clear_rows words.  A word that
// began before the part leaves its sum in parts[a][0], one that began here and
// goes on behind the part in parts[a][1], all others are done.
__global__ void __launch_bounds__(SUM_THREADS) embedding_sum_kernel(const Entry* sorted,
                                                                   const int32_t* start, int v, int part,
                                                                   long long n_parts, int slices, int clear_rows, int h,
                                                                   float scale, const __nv_bfloat16* dOut,
                                                                   float* dE, int accumulate, float* parts,
                                                                   int32_t* counters) {
    __shared__ Entry mine[MAX_PART + 2];  // with the neighbours of both ends
    __shared__ int last;
    static_assert(sizeof(mine) >= (MAX_CLEAR + 1) * sizeof(int32_t), "");
    pdl_trigger();
    pdl_wait();
    const long long a = blockIdx.x / slices, n = start[v], from = a * part;
    const int slice = blockIdx.x % slices;
    if (a >= n_parts) {
        const long long first = (blockIdx.x - n_parts * slices) * clear_rows;
        clear_words(start, first, static_cast<int>(min(static_cast<long long>(clear_rows), v - first)), h, dE, &mine[0].word);
        return;
    }
    const int tokens = static_cast<int>(min(static_cast<long long>(part), n - from));
    if (tokens <= 0) return;
    for (int k = threadIdx.x; k < tokens + 2; k += blockDim.x) {
        const long long i = from + k - 1;
        mine[k] = i >= 0 && i < n ? sorted[i] : Entry{-1, 0};
    }
    __syncthreads();
    const int c = slice * blockDim.x + threadIdx.x;
    const bool in = c < h >> 3;
    // The words that this part's borders cut, and the parts that they span: the
    // first one's sum is part of a word that came, the last one's of a word that
    // goes on (one word, one sum).
    bool ends[2] = {mine[0].word == mine[1].word, mine[tokens].word == mine[tokens + 1].word};
    if (ends[0] && mine[1].word == mine[tokens].word) ends[1] = false;
    int2 span[2] = {};
#pragma unroll
    for (int k = 0; k < 2; ++k)
        if (ends[k]) span[k] = make_int2(start[mine[k ? tokens : 1].word], start[mine[k ? tokens : 1].word + 1]);
    float s[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    bool came = mine[0].word == mine[1].word;
    for (int at = 0; in && at < tokens; at += SUM_LOADS) {
        uint4 u[SUM_LOADS];
#pragma unroll
        for (int k = 0; k < SUM_LOADS; ++k) {
            const int i = min(at + k, tokens - 1);  // loads past the end repeat the last row
            u[k] = reinterpret_cast<const uint4*>(dOut + static_cast<long long>(mine[i + 1].at) * h)[c];
        }
#pragma unroll
        for (int k = 0; k < SUM_LOADS; ++k) {
            const int i = at + k;
            if (i >= tokens) break;
            float f[8];
            unpack8(u[k], f);
#pragma unroll
            for (int e = 0; e < 8; ++e) s[e] += f[e];
            const int word = mine[i + 1].word;
            const bool more = mine[i + 2].word == word;
            if (more && i + 1 < tokens) continue;
            if (came || more) store_sum(parts + (2 * a + !came) * h, c, s, 1.0f, 0);
            else store_sum(dE + static_cast<long long>(word) * h, c, s, scale, accumulate);
            came = false;
#pragma unroll
            for (int e = 0; e < 8; ++e) s[e] = 0.0f;
        }
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        if (!ends[k]) continue;
        const int word = mine[k ? tokens : 1].word;
        const long long first = span[k].x / part, past = (span[k].y - 1) / part;
        __threadfence();  // this thread's sums, before the count that announces them
        __syncthreads();
        if (threadIdx.x == 0) last = atomicAdd(counters + first * slices + slice, 1) == past - first;
        __syncthreads();
        if (!last || !in) continue;
        __threadfence();
        float t[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        for (long long b0 = first; b0 <= past; b0 += SUM_LOADS) {
            float4 x[SUM_LOADS], y[SUM_LOADS];
#pragma unroll
            for (int k = 0; k < SUM_LOADS; ++k) {
                const long long b = b0 + k;
                const float4* p = reinterpret_cast<const float4*>(parts + (2 * b + (b == first)) * h) + 2 * c;
                x[k] = b <= past ? __ldcg(p) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                y[k] = b <= past ? __ldcg(p + 1) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            }
#pragma unroll
            for (int k = 0; k < SUM_LOADS; ++k) {
                t[0] += x[k].x, t[1] += x[k].y, t[2] += x[k].z, t[3] += x[k].w;
                t[4] += y[k].x, t[5] += y[k].y, t[6] += y[k].z, t[7] += y[k].w;
            }
        }
        store_sum(dE + static_cast<long long>(word) * h, c, t, scale, accumulate);
    }
}

constexpr int PART_CTAS = 1024;
// Sorted tokens of a part: so many that about PART_CTAS CTAs (parts times slices of
// columns) share the work, between 8 and MAX_PART.
int part_tokens(int64_t M, int h) {
    const int64_t slices = (h / 8 + SUM_THREADS - 1) / SUM_THREADS;
    int64_t part = 8;
    while (part < MAX_PART && part * PART_CTAS < M * slices) part *= 2;
    return static_cast<int>(part);
}

// ------------------------------------------------------------ loss and its gradient

// Running maximum and sum of 2^((z - max) log2 e).  A maximum of -inf (nothing
// yet, or masked logits alone) counts as 0, so that no difference is NaN.
struct MS {
    float m, s;
};
__device__ __forceinline__ float finite_max(float m) { return m == -INFINITY ? 0.0f : m; }
__device__ __forceinline__ MS ms_merge(MS a, MS b) {
    const float m = fmaxf(a.m, b.m), n = finite_max(m);
    return {m, a.s * ex2f((a.m - n) * LOG2E) + b.s * ex2f((b.m - n) * LOG2E)};
}

// The sum runs over the other words than the label, so that neither the label's
// gradient (p - 1) nor a small loss comes from a difference: with n the row's
// largest logit, o = sum_{j != y} e^{z_j - n} and s = o + e^{z_y - n},
//   loss = n - z_y + log s  (log(1 + o) where the label is the largest),
//   dz_j = dloss e^{z_j - n} / s,  dz_y = -dloss o / s.
struct RowEnd {
    float n, others, sum;
};
// y: the label's logit; most: the largest other one; others(n): their sum of e^{z - n}.
template <typename F>
__device__ __forceinline__ RowEnd row_end(float y, float most, F&& others) {
    const float n = finite_max(fmaxf(most, y)), o = others(n);
    return {n, o, o + ex2f((y - n) * LOG2E)};
}
__device__ __forceinline__ float loss_of(const RowEnd& r, float y) {
    if (r.sum != r.sum) return r.sum;
    return r.n == y ? log1pf(r.others) : (r.n - y) + logf(r.sum);
}

// A label outside the vocabulary: ignored (loss and gradient 0) or wrong (NaN).
__device__ __forceinline__ uint32_t fill_of(int label) { return label == -100 ? 0u : 0x7fc07fc0u; }

// Rows of any length: one CTA a token, which reads the row twice.
constexpr int LOSS_THREADS = 512;

__global__ void __launch_bounds__(LOSS_THREADS) loss_long_kernel(const __nv_bfloat16* logits, int v,
                                                                 const int32_t* labels,
                                                                 const float* dloss, float* loss,
                                                                 __nv_bfloat16* dlogits) {
    __shared__ MS red[LOSS_THREADS / 32];
    __shared__ float label_z;
    pdl_trigger();
    pdl_wait();
    const long long m = blockIdx.x;
    const int label = labels[m];
    const uint4* z = reinterpret_cast<const uint4*>(logits + m * v);
    uint4* d = reinterpret_cast<uint4*>(dlogits + m * v);
    const int nv = v >> 3;
    if (label < 0 || label >= v) {
        const uint32_t fill = fill_of(label);
        for (int c = threadIdx.x; c < nv; c += LOSS_THREADS) d[c] = make_uint4(fill, fill, fill, fill);
        if (threadIdx.x == 0) loss[m] = __uint_as_float(fill & 0xffff0000u);
        return;
    }
    MS acc = {-INFINITY, 0.0f};
    for (int c = threadIdx.x; c < nv; c += LOSS_THREADS) {
        float x[8];
        unpack8(z[c], x);
        if (c == label >> 3) {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (e == (label & 7)) {
                    label_z = x[e];
                    x[e] = -INFINITY;
                }
        }
        float most = acc.m;
#pragma unroll
        for (int e = 0; e < 8; ++e) most = fmaxf(most, x[e]);
        const float n = finite_max(most);
        float s = acc.s * ex2f((acc.m - n) * LOG2E);
#pragma unroll
        for (int e = 0; e < 8; ++e) s += ex2f((x[e] - n) * LOG2E);
        acc = {most, s};
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        acc = ms_merge(acc, MS{__shfl_xor_sync(0xffffffffu, acc.m, o), __shfl_xor_sync(0xffffffffu, acc.s, o)});
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = acc;
    __syncthreads();
    acc = red[0];
    for (int k = 1; k < LOSS_THREADS / 32; ++k) acc = ms_merge(acc, red[k]);
    const RowEnd r = row_end(label_z, acc.m, [&](float n) { return acc.s * ex2f((acc.m - n) * LOG2E); });
    const float by = __fdividef(dloss ? dloss[m] : 1.0f, r.sum);
    if (threadIdx.x == 0) loss[m] = loss_of(r, label_z);
    for (int c = threadIdx.x; c < nv; c += LOSS_THREADS) {
        float x[8];
        unpack8(z[c], x);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            x[e] = ex2f((x[e] - r.n) * LOG2E) * by;
            if (c == label >> 3 && e == (label & 7)) x[e] = -r.others * by;
        }
        d[c] = pack8(x);
    }
}

// Rows that a cluster of CTAs holds in shared memory: LOSS_VPT 16-byte pieces a
// thread and row, which that thread alone copies and reads, so that no barrier
// guards them; each logit is read once and each gradient written once.  Each
// warp's maximum and sum, and the label's logit, go to every CTA of the cluster by
// st.async, counted on the receiver's mbarrier.  A row's gradients are computed after the next row's sums,
// so nothing waits for the exchange: with a wait between a row's two passes 8192 x
// 128256 took 843 us, with a cluster barrier there (whose release waits for the
// last row's stores) about as much.
// Four slots in turn: a CTA that sends row r's sums has all sums of row r - 2, whose
// senders had finished with row r - 4, so its slot is free everywhere.
constexpr int LOSS_VPT = 8, LOSS_ROW_THREADS = 256, LOSS_CTAS = 2, LOSS_STAGES = 3, LOSS_SLOTS = 4;
constexpr int LOSS_PIECES = LOSS_VPT * LOSS_ROW_THREADS, LOSS_RANKS = 16;

__device__ __forceinline__ void copy_piece(uint32_t to, const void* from) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {  // all groups of this thread but the last N
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ uint32_t max_bf16x2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("max.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
__device__ __forceinline__ float warp_max(float x) {
    float d;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(d) : "f"(x));
    return d;
}
__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

// mbar_wait for what other CTAs of the cluster stored.
constexpr uint64_t LOSS_TIMEOUT_NS = 2000000000ull;

__device__ __forceinline__ bool cluster_try_wait(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0u;
}
__device__ __forceinline__ bool cluster_wait_bar(uint32_t bar, uint32_t parity, volatile int* abort_flag) {
    if (cluster_try_wait(bar, parity)) return true;
    const uint64_t t0 = globaltimer_ns();
    while (true) {
#pragma unroll 1
        for (int i = 0; i < 32; ++i)
            if (cluster_try_wait(bar, parity)) return true;
        if (*abort_flag) return false;
        if (globaltimer_ns() - t0 > LOSS_TIMEOUT_NS) {
            *abort_flag = 1;
            return false;
        }
    }
}

struct LossRow {
    int label;
    float up;  // the loss's gradient
};

// 2^(z scale - shift), two logits at a time, for e^(z - n) = 2^((z - n) log2 e):
// shift is n scale rounded, and what it lacks goes into the sums as `rest`, exactly.
// Above 2^23 logits that differ are 2^15 apart: any scale serves there, and 1 does
// without rounding.
struct Power {
    uint64_t scale, shift;
    float rest;
    __device__ __forceinline__ explicit Power(float n) {
        const float c = fabsf(n) < 0x1p23f ? LOG2E : 1.0f, s = n * c;
        scale = f2_pack(c, c);
        shift = f2_pack(-s, -s);
        rest = c == 1.0f ? 1.0f : ex2f(-fmaf(n, c, -s));
    }
    __device__ __forceinline__ uint64_t operator()(uint32_t word) const {
        float a, b;
        f2_unpack(f2_fma(f2_pack(__uint_as_float(word << 16), __uint_as_float(word & 0xffff0000u)), scale, shift), a, b);
        return f2_pack(ex2f(a), ex2f(b));
    }
};

__global__ void __launch_bounds__(LOSS_ROW_THREADS, LOSS_CTAS) loss_kernel(const __nv_bfloat16* logits, long long M, int v,
                                                                           int per, int ranks,
                                                                           const int32_t* labels,
                                                                           const float* dloss,
                                                                           float* loss, __nv_bfloat16* dlogits) {
    __shared__ MS slots[LOSS_SLOTS][LOSS_RANKS * LOSS_ROW_THREADS / 32 + 1];  // the warps', the label's
    __shared__ __align__(8) uint64_t arrived[LOSS_SLOTS];
    __shared__ int abort_flag, no_abort;
    extern __shared__ uint4 ring[];  // [LOSS_STAGES][LOSS_VPT][threads]
    pdl_trigger();
    const int rank = ranks > 1 ? static_cast<int>(cluster_ctarank()) : 0;
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, warps = blockDim.x >> 5, entries = ranks * warps;
    // This warp's pieces of a row: lo + lane, lo + 32 + lane, ... up to `pieces` (none where <= 0).
    const int lo = rank * per + w * 32 * LOSS_VPT, pieces = min(rank * per + per, v >> 3) - lo;
    const long long step = gridDim.x / ranks;
    if (threadIdx.x == 0) {
        for (int k = 0; k < LOSS_SLOTS; ++k) mbar_init(smem_u32(&arrived[k]), 1);
        abort_flag = no_abort = 0;
        fence_barrier_init();
    }
    const int stage_pieces = LOSS_VPT * blockDim.x;
    for (int i = threadIdx.x; i < LOSS_STAGES * stage_pieces; i += blockDim.x)
        ring[i] = make_uint4(0xff80ff80u, 0xff80ff80u, 0xff80ff80u, 0xff80ff80u);  // -inf behind the row's end
    if (ranks > 1) cluster_sync_all();  // the others run, before anything is stored there
    else __syncthreads();
    pdl_wait();

    auto label_at = [&](long long m) { return m < M ? labels[m] : -100; };
    auto exists = [&](int label) { return label >= 0 && label < v; };
    // A row's copies and scalars; its label has been read a row before, so that
    // nothing here waits for memory.
    auto load = [&](long long m, int label, int stage) {
        LossRow row = {label, 0.0f};
        if (exists(label)) {
            row.up = dloss ? dloss[m] : 1.0f;
            const uint4* z = reinterpret_cast<const uint4*>(logits + m * v) + lo + lane;
            const uint32_t to = smem_u32(ring + stage * stage_pieces + threadIdx.x);
#pragma unroll
            for (int i = 0; i < LOSS_VPT; ++i)
                if (32 * i + lane < pieces) copy_piece(to + i * blockDim.x * 16, z + 32 * i);
        }
        copies_commit();
        return row;
    };
    // Where the label's logit lies, if it is this thread's; else -1.
    auto own_piece = [&](int label) {
        const int own = (label >> 3) - lo;
        return own >= 0 && own < min(pieces, 32 * LOSS_VPT) && (own & 31) == lane ? own : -1;
    };
    // First pass: the sums of the other words' powers, on their way to every CTA.
    auto send = [&](const LossRow& row, int stage, unsigned number) {
        uint4* here = ring + stage * stage_pieces + threadIdx.x;
        const int own = own_piece(row.label);
        MS* slot = slots[number % LOSS_SLOTS];
        const uint32_t bar = smem_u32(&arrived[number % LOSS_SLOTS]);
        if (ranks > 1 && threadIdx.x == 0) mbar_arrive_expect_tx(bar, (entries + 1) * sizeof(MS));
        auto put = [&](int at, float a, float b) {
            if (ranks == 1) {
                if (lane == 0) slot[at] = {a, b};
            } else if (lane < ranks) {
                asm volatile(
                    "st.async.shared::cluster.mbarrier::complete_tx::bytes.v2.f32 [%0], {%1, %2}, [%3];" ::"r"(
                        mapa_shared(smem_u32(slot + at), lane)),
                    "f"(a), "f"(b), "r"(mapa_shared(bar, lane))
                    : "memory");
            }
        };
        // The label's logit goes round by itself and leaves the sum: -inf in its place.
        const unsigned owner = __ballot_sync(0xffffffffu, own >= 0);
        if (owner) {
            float y = 0.0f;
            if (own >= 0) {
                uint16_t* at = reinterpret_cast<uint16_t*>(here + (own >> 5) * blockDim.x) + (row.label & 7);
                y = __uint_as_float(static_cast<uint32_t>(*at) << 16);
                *at = 0xff80u;
            }
            put(entries, __shfl_sync(0xffffffffu, y, __ffs(owner) - 1), 0.0f);
        }
        uint4 u[LOSS_VPT];
        uint32_t top = 0xff80ff80u;
#pragma unroll
        for (int i = 0; i < LOSS_VPT; ++i) {
            u[i] = here[i * blockDim.x];
            top = max_bf16x2(top, max_bf16x2(max_bf16x2(u[i].x, u[i].y), max_bf16x2(u[i].z, u[i].w)));
        }
        const float2 tops = unpack_bf16x2(top);
        const float most = warp_max(fmaxf(tops.x, tops.y));
        const Power power(finite_max(most));
        uint64_t s0 = f2_pack(0.0f, 0.0f), s1 = s0;
#pragma unroll
        for (int i = 0; i < LOSS_VPT; ++i) {
            s0 = f2_add(s0, power(u[i].x));
            s1 = f2_add(s1, power(u[i].y));
            s0 = f2_add(s0, power(u[i].z));
            s1 = f2_add(s1, power(u[i].w));
        }
        float a, b;
        f2_unpack(f2_add(s0, s1), a, b);
        const float sum = warp_sum(a + b) * power.rest;
        put(rank * warps + w, most, sum);
        if (ranks == 1) __syncthreads();
    };
    // Second pass: the row's loss and gradients.  False where a wait gave up.
    auto finish = [&](const LossRow& row, long long m, int stage, unsigned number) {
        uint4* d = reinterpret_cast<uint4*>(dlogits + m * v) + lo + lane;
        if (!exists(row.label)) {
            const uint32_t fill = fill_of(row.label);
#pragma unroll
            for (int i = 0; i < LOSS_VPT; ++i)
                if (32 * i + lane < pieces) d[32 * i] = make_uint4(fill, fill, fill, fill);
            if (rank == 0 && threadIdx.x == 0) loss[m] = __uint_as_float(fill & 0xffff0000u);
            return true;
        }
        if (ranks > 1 && !__all_sync(0xffffffffu, cluster_wait_bar(smem_u32(&arrived[number % LOSS_SLOTS]),
                                                                   number / LOSS_SLOTS & 1, &abort_flag)))
            return false;
        const MS* slot = slots[number % LOSS_SLOTS];
        MS all[LOSS_RANKS * LOSS_ROW_THREADS / 32 / 32];
        float highest = -INFINITY;
#pragma unroll
        for (int k = 0; k < LOSS_RANKS * LOSS_ROW_THREADS / 32 / 32; ++k) {
            all[k] = 32 * k + lane < entries ? slot[32 * k + lane] : MS{-INFINITY, 0.0f};
            highest = fmaxf(highest, all[k].m);
        }
        const float y = slot[entries].m;
        const RowEnd r = row_end(y, warp_max(highest), [&](float n) {
            float s = 0.0f;
#pragma unroll
            for (int k = 0; k < LOSS_RANKS * LOSS_ROW_THREADS / 32 / 32; ++k)
                if (32 * k < entries) s += all[k].s * ex2f((all[k].m - n) * LOG2E);
            return warp_sum(s);
        });
        const float scale = __fdividef(row.up, r.sum);
        if (rank == 0 && threadIdx.x == 0) loss[m] = loss_of(r, y);
        const Power power(r.n);
        const uint64_t by = f2_pack(scale * power.rest, scale * power.rest);
        auto grad = [&](uint32_t word) {
            float lo_z, hi_z;
            f2_unpack(f2_mul(power(word), by), lo_z, hi_z);
            return pack_bf16x2(lo_z, hi_z);
        };
        const uint4* here = ring + stage * stage_pieces + threadIdx.x;
#pragma unroll
        for (int i = 0; i < LOSS_VPT; ++i) {
            const uint4 u = here[i * blockDim.x];
            if (32 * i + lane < pieces) d[32 * i] = make_uint4(grad(u.x), grad(u.y), grad(u.z), grad(u.w));
        }
        // The label's gradient over what its piece's store left in its place.
        const int own = own_piece(row.label);
        if (own >= 0) reinterpret_cast<__nv_bfloat16*>(d + (own & ~31))[row.label & 7] = __float2bfloat16_rn(-r.others * scale);
        return true;
    };

    long long m = blockIdx.x / ranks;
    LossRow last = {-100, 0.0f}, row = load(m, label_at(m), 0), next = load(m + step, label_at(m + step), 1);
    int label = label_at(m + 2 * step), stage = 0;
    unsigned sent = 0;  // rows whose sums went round
    bool ok = true;
    // Row m's sums, then the gradients of the row before it.
    for (; m < M + step; m += step) {
        const bool here = m < M && exists(row.label);
        copies_wait<1>();
        const int before = stage == 0 ? LOSS_STAGES - 1 : stage - 1;
        if (here) send(row, stage, sent);
        if (m >= step) {  // (no row before the first one)
            ok = finish(last, m - step, before, sent - 1);
            if (!ok) break;
        }
        if (here) ++sent;
        const int now = label;
        label = label_at(m + 3 * step);
        last = row;
        row = next;
        next = load(m + 2 * step, now, before);
        stage = stage == LOSS_STAGES - 1 ? 0 : stage + 1;
    }
    if (!ok) {  // the losses of the rows left say so
        copies_wait<0>();
        for (long long r = m - step; rank == 0 && threadIdx.x == 0 && r < M; r += step) loss[r] = __int_as_float(0x7fc00000);
    }
    if (ranks > 1) {
        __syncwarp();
        cluster_sync_all();  // nothing more is stored in another CTA's shared memory
        if (!ok)             // what was on its way here has arrived, as far as it comes
            for (unsigned k = 0; k < LOSS_SLOTS; ++k) {
                const unsigned number = sent + k >= 1 ? sent + k - 1 : 0;
                cluster_wait_bar(smem_u32(&arrived[number % LOSS_SLOTS]), number / LOSS_SLOTS & 1, &no_abort);
            }
    }
}

size_t loss_ring_bytes(int threads) { return static_cast<size_t>(LOSS_STAGES) * LOSS_VPT * threads * sizeof(uint4); }

// Clusters of `ranks` CTAs of loss_kernel that the current device holds at once; 0
// when they do not fit at all.
int loss_clusters(int ranks, int threads) {
    static int counts[64][5][LOSS_ROW_THREADS / 32] = {};
    int dev = 0, log = 0;
    while (1 << log < ranks) ++log;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
    int& count = counts[dev][log][threads / 32 - 1];
    if (!count) {
        int n = 0;
        cudaLaunchConfig_t cfg;
        memset(&cfg, 0, sizeof(cfg));
        cfg.gridDim = dim3(ranks * 64);
        cfg.blockDim = dim3(threads);
        cfg.dynamicSmemBytes = loss_ring_bytes(threads);
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = ranks;
        attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        if (cudaFuncSetAttribute(loss_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess ||
            cudaFuncSetAttribute(loss_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 static_cast<int>(loss_ring_bytes(LOSS_ROW_THREADS))) != cudaSuccess ||
            cudaOccupancyMaxActiveClusters(&n, loss_kernel, &cfg) != cudaSuccess)
            n = 0;
        cudaGetLastError();
        count = n > 0 ? n : -1;
    }
    return count > 0 ? count : 0;
}

int check(const char* what, std::string* err) {
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) {
        if (err) *err = std::string(what) + ": " + cudaGetErrorString(e);
        return TP_ERR_CUDA;
    }
    return TP_OK;
}

}  // namespace

namespace tpi {

int vocab_embedding_scaled_launch(const int32_t* ids, int64_t M, const void* E, int64_t v, int h, float scale, void* out,
                                  cudaStream_t stream, std::string* err) {
    if (M == 0) return TP_OK;
    launch_pdl(embedding_scaled_kernel, dim3((unsigned)((M + EMB_WARPS - 1) / EMB_WARPS)), dim3(EMB_WARPS * 32), 0, stream,
               ids, static_cast<long long>(M), static_cast<const __nv_bfloat16*>(E), static_cast<long long>(v), h, scale,
               static_cast<__nv_bfloat16*>(out));
    return check("scaled embedding kernel", err);
}

// Scratch: where each word's tokens start, a counter for each part and slice of
// columns, the sorted tokens, and two partial sums a part.
struct EmbeddingScratch {
    int64_t parts, slices;
    int part, threads;
    size_t counters, sorted, sums, bytes;
    EmbeddingScratch(int64_t M, int64_t v, int h) {
        part = part_tokens(M, h);
        threads = std::min(SUM_THREADS, (h / 8 + 31) / 32 * 32);
        parts = (M + part - 1) / part;
        slices = (h / 8 + threads - 1) / threads;
        auto after = [](size_t at, int64_t n, size_t each) { return (at + static_cast<size_t>(n) * each + 15) / 16 * 16; };
        counters = after(0, v + 1, sizeof(int32_t));
        sorted = after(counters, parts * slices, sizeof(int32_t));
        sums = after(sorted, M, sizeof(Entry));
        bytes = after(sums, parts > 1 ? parts * 2 * h : 0, sizeof(float));
    }
};
size_t vocab_embedding_bwd_scratch_bytes(int64_t M, int64_t v, int h) { return EmbeddingScratch(M, v, h).bytes; }

int vocab_embedding_bwd_launch(const int32_t* ids, int64_t M, int64_t v, int h, float scale, const void* dOut, float* dE,
                               int accumulate, void* scratch, cudaStream_t stream, std::string* err) {
    const EmbeddingScratch at(M, v, h);
    char* base = static_cast<char*>(scratch);
    int32_t *start = reinterpret_cast<int32_t*>(base), *counters = reinterpret_cast<int32_t*>(base + at.counters);
    Entry* sorted = reinterpret_cast<Entry*>(base + at.sorted);
    const int warps = static_cast<int>(std::min<int64_t>(std::max<int64_t>((M + 32 * SORT_LOADS - 1) / (32 * SORT_LOADS), BINS / 32),
                                                         MAX_SORT_WARPS));
    launch_pdl(sort_tokens_kernel, dim3((unsigned)((v + BINS - 1) / BINS)), dim3(warps * 32),
               static_cast<size_t>(warps) * BINS * sizeof(int32_t), stream, ids,
               static_cast<long long>(M), static_cast<int>(v), sorted, start, counters,
               static_cast<long long>(at.parts * at.slices));
    const int rc = check("token sort kernel", err);
    const int64_t clear_rows = std::min<int64_t>(std::max<int64_t>(1, CLEAR_BYTES / 4 / h), MAX_CLEAR);
    const int64_t grid = at.parts * at.slices + (accumulate ? 0 : (v + clear_rows - 1) / clear_rows);
    if (rc || grid == 0) return rc;
    launch_pdl(embedding_sum_kernel, dim3((unsigned)grid), dim3(at.threads), 0, stream, static_cast<const Entry*>(sorted),
               static_cast<const int32_t*>(start), static_cast<int>(v), at.part, static_cast<long long>(at.parts),
               static_cast<int>(at.slices), static_cast<int>(clear_rows), h, scale,
               static_cast<const __nv_bfloat16*>(dOut), dE, accumulate, reinterpret_cast<float*>(base + at.sums), counters);
    return check("embedding gradient kernel", err);
}

int vocab_loss_launch(const void* logits, int64_t M, int64_t v, const int32_t* labels, const float* dloss, float* loss,
                      void* dlogits, cudaStream_t stream, std::string* err) {
    if (M == 0) return TP_OK;
    const __nv_bfloat16* z = static_cast<const __nv_bfloat16*>(logits);
    __nv_bfloat16* d = static_cast<__nv_bfloat16*>(dlogits);
    const int64_t nv = v / 8;
    int ranks = 1;
    while (ranks < LOSS_RANKS && nv > static_cast<int64_t>(ranks) * LOSS_PIECES) ranks *= 2;
    const int64_t per = (nv + ranks - 1) / ranks;
    const int threads = static_cast<int>(std::min<int64_t>((per + 32 * LOSS_VPT - 1) / (32 * LOSS_VPT) * 32, LOSS_ROW_THREADS));
    const int64_t clusters = per > LOSS_PIECES ? 0 : loss_clusters(ranks, threads);
    if (clusters < 1) {
        launch_pdl(loss_long_kernel, dim3((unsigned)M), dim3(LOSS_THREADS), 0, stream, z, static_cast<int>(v), labels, dloss,
                   loss, d);
        return check("loss kernel", err);
    }
    cudaLaunchConfig_t cfg;
    memset(&cfg, 0, sizeof(cfg));
    cfg.gridDim = dim3((unsigned)(std::min<int64_t>(M, clusters) * ranks));
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = loss_ring_bytes(threads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    pdl_attribute(attr[0]);
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = ranks;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    cudaLaunchKernelEx(&cfg, loss_kernel, z, static_cast<long long>(M), static_cast<int>(v), static_cast<int>(per), ranks,
                       labels, dloss, loss, d);
    return check("loss kernel", err);
}

}  // namespace tpi
