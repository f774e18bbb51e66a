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

// One warp per token: out = scale * E[id] (rounded once), or zeros.
constexpr int EMB_WARPS = 8;

__global__ void __launch_bounds__(EMB_WARPS * 32) embedding_scaled_kernel(const int32_t* __restrict__ ids, long long M,
                                                                         const __nv_bfloat16* __restrict__ E, long long v,
                                                                         int h, float scale, __nv_bfloat16* __restrict__ out) {
    pdl_trigger();
    pdl_wait();
    const long long m = static_cast<long long>(blockIdx.x) * EMB_WARPS + (threadIdx.x >> 5);
    if (m >= M) return;
    const long long id = ids[m];
    const bool owned = id >= 0 && id < v;
    const uint4* src = reinterpret_cast<const uint4*>(E + (owned ? id : 0) * h);
    uint4* dst = reinterpret_cast<uint4*>(out + m * h);
    for (int c = threadIdx.x & 31; c < (h >> 3); c += 32) {
        float f[8];
        unpack8(owned ? src[c] : make_uint4(0, 0, 0, 0), f);
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = owned ? f[e] * scale : 0.0f;
        dst[c] = pack8(f);
    }
}

// ------------------------------------------------------------ embedding gradient

// Three launches, no atomics on values, the same bits every time:
//  1. tokens sorted by word, and zeros for words without a token;
//  2. the sorted tokens in parts of equal length, summed by word; a word that a
//     part's border cuts leaves partial sums;
//  3. the words that borders cut, their partial sums added in order.
// Parts of equal length keep a frequent word (in text, one token in ten is the
// same one) from being one CTA's work.

// Sorting: a CTA owns BINS words and looks through all ids: it counts the
// tokens of words below its own (its place in the order) and of each of its
// own, then puts the positions down word by word.  Every warp takes a
// contiguous part of the tokens and has counters of its own, so the positions
// of a word come out ascending whatever the order of the work.
constexpr int BINS = 128, SORT_WARPS = 32, SORT_LOADS = 8;

struct Entry {
    int32_t word, at;  // a token's word and its position
};

// Calls f(id, position) for this lane's tokens of [from, to), 32 consecutive
// ones a warp and call; -1 past the end.
template <typename F>
__device__ __forceinline__ void for_ids(const int32_t* __restrict__ ids, long long from, long long to, F&& f) {
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

__global__ void __launch_bounds__(SORT_WARPS * 32) sort_tokens_kernel(const int32_t* __restrict__ ids, long long M, int v,
                                                                     Entry* __restrict__ sorted, int32_t* __restrict__ valid,
                                                                     int h, float* __restrict__ clear) {
    __shared__ int32_t count[SORT_WARPS][BINS];
    __shared__ int32_t below[SORT_WARPS], sums[BINS / 32], tokens[BINS];
    pdl_trigger();
    pdl_wait();
    const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int lo = blockIdx.x * BINS, bins = min(BINS, v - lo);
    for (int b = lane; b < BINS; b += 32) count[w][b] = 0;
    __syncwarp();
    const long long part = ((M + SORT_WARPS - 1) / SORT_WARPS + 31) / 32 * 32;
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
        for (int k = 0; k < SORT_WARPS; ++k) {
            const int n = count[k][threadIdx.x];
            count[k][threadIdx.x] = total;
            total += n;
            base += below[k];
        }
        tokens[threadIdx.x] = total;
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
        for (int k = 0; k < SORT_WARPS; ++k) count[k][threadIdx.x] += base;
        if (lo + static_cast<int>(threadIdx.x) == v - 1) *valid = base + total;
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
    if (!clear) return;
    for (int b = w; b < bins; b += SORT_WARPS) {
        if (tokens[b]) continue;
        float4* row = reinterpret_cast<float4*>(clear + (static_cast<long long>(lo) + b) * h);
        for (int c = lane; c < h >> 2; c += 32) row[c] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    }
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

// Sorted tokens [a part, (a + 1) part) for one slice of columns.  A word that
// began before the part leaves its sum in parts[a][0], one that began here and
// goes on behind the part in parts[a][1], all others are done.
__global__ void __launch_bounds__(SUM_THREADS) embedding_sum_kernel(const Entry* __restrict__ sorted,
                                                                   const int32_t* __restrict__ valid, int part, int h,
                                                                   float scale, const __nv_bfloat16* __restrict__ dOut,
                                                                   float* dE, int accumulate, float* __restrict__ parts) {
    __shared__ Entry mine[MAX_PART + 2];  // with the neighbours of both ends
    pdl_trigger();
    pdl_wait();
    const long long a = blockIdx.x, n = *valid, from = a * part;
    const int tokens = static_cast<int>(min(static_cast<long long>(part), n - from));
    if (tokens <= 0) return;
    for (int k = threadIdx.x; k < tokens + 2; k += blockDim.x) {
        const long long i = from + k - 1;
        mine[k] = i >= 0 && i < n ? sorted[i] : Entry{-1, 0};
    }
    __syncthreads();
    const int c = blockIdx.y * blockDim.x + threadIdx.x;
    if (c >= h >> 3) return;
    float s[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    bool came = mine[0].word == mine[1].word;
    for (int at = 0; at < tokens; at += SUM_LOADS) {
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
}

// The word that began in part a and goes on behind it: its parts in order.
__global__ void __launch_bounds__(SUM_THREADS) embedding_join_kernel(const Entry* __restrict__ sorted,
                                                                    const int32_t* __restrict__ valid, int part, int h,
                                                                    float scale, float* dE, int accumulate,
                                                                    const float* __restrict__ parts) {
    pdl_trigger();
    pdl_wait();
    const long long a = blockIdx.x, n = *valid, end = (a + 1) * part;
    if (end >= n) return;
    const int word = sorted[end].word;
    if (sorted[end - 1].word != word) return;
    if (a && sorted[a * part].word == word && sorted[a * part - 1].word == word) return;  // it began before
    long long more = 0;  // parts that begin inside the word
    for (long long at = end;; at += static_cast<long long>(part) * blockDim.x) {
        const long long i = at + static_cast<long long>(part) * threadIdx.x;
        const int here = __syncthreads_count(i < n && sorted[i].word == word);
        more += here;
        if (here < static_cast<int>(blockDim.x)) break;
    }
    const int c = blockIdx.y * blockDim.x + threadIdx.x;
    if (c >= h >> 3) return;
    float s[8];
    const float4* first = reinterpret_cast<const float4*>(parts + (2 * a + 1) * h) + 2 * c;
    float4 x = first[0], y = first[1];
    s[0] = x.x, s[1] = x.y, s[2] = x.z, s[3] = x.w, s[4] = y.x, s[5] = y.y, s[6] = y.z, s[7] = y.w;
#pragma unroll 4
    for (long long k = 1; k <= more; ++k) {
        const float4* p = reinterpret_cast<const float4*>(parts + 2 * (a + k) * h) + 2 * c;
        x = p[0], y = p[1];
        s[0] += x.x, s[1] += x.y, s[2] += x.z, s[3] += x.w, s[4] += y.x, s[5] += y.y, s[6] += y.z, s[7] += y.w;
    }
    store_sum(dE + static_cast<long long>(word) * h, c, s, scale, accumulate);
}

// Sorted tokens of a part: so many that about 2048 CTAs (parts times slices of
// columns) share the work, between 8 and MAX_PART.
int part_tokens(int64_t M, int h) {
    const int64_t slices = (h / 8 + SUM_THREADS - 1) / SUM_THREADS;
    int64_t part = 8;
    while (part < MAX_PART && part * 2048 < M * slices) part *= 2;
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

// One CTA per token.  The sum runs over the other words than the label, so that
// neither the label's gradient (p - 1) nor a small loss comes from a difference:
//   r = (sum_{j != y} e^{z_j}) / e^{z_y},  loss = log(1 + r),
//   dz_y = -dloss r / (1 + r),  dz_j = dloss e^{z_j - z_y} / (1 + r).
constexpr int LOSS_THREADS = 512;

__global__ void __launch_bounds__(LOSS_THREADS) loss_kernel(const __nv_bfloat16* logits, int v,
                                                            const int32_t* __restrict__ labels,
                                                            const float* __restrict__ dloss, float* __restrict__ loss,
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
        const bool ignored = label == -100;
        const uint32_t fill = ignored ? 0u : 0x7fc07fc0u;
        for (int c = threadIdx.x; c < nv; c += LOSS_THREADS) d[c] = make_uint4(fill, fill, fill, fill);
        if (threadIdx.x == 0) loss[m] = ignored ? 0.0f : __int_as_float(0x7fc00000);
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
    const float y = label_z, most = fmaxf(acc.m, y), n = finite_max(most);
    const float others = acc.s * ex2f((acc.m - n) * LOG2E), mine = ex2f((y - n) * LOG2E), sum = others + mine;
    const float up = dloss ? dloss[m] : 1.0f, by = up / sum;
    if (threadIdx.x == 0) loss[m] = y >= acc.m && mine == 1.0f ? log1pf(others) : (n - y) + logf(sum);
    for (int c = threadIdx.x; c < nv; c += LOSS_THREADS) {
        float x[8];
        unpack8(z[c], x);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            x[e] = ex2f((x[e] - n) * LOG2E) * by;
            if (c == label >> 3 && e == (label & 7)) x[e] = -others * by;
        }
        d[c] = pack8(x);
    }
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

// Scratch: the number of tokens whose word exists, the sorted tokens, and two
// partial sums a part.
size_t vocab_embedding_bwd_scratch_bytes(int64_t M, int64_t v, int h) {
    const int64_t part = part_tokens(M, h), n = (M + part - 1) / part;
    return 16 + static_cast<size_t>((M + 1) / 2 * 2) * sizeof(Entry) + static_cast<size_t>(n > 1 ? n : 0) * 2 * h * sizeof(float);
}

int vocab_embedding_bwd_launch(const int32_t* ids, int64_t M, int64_t v, int h, float scale, const void* dOut, float* dE,
                               int accumulate, void* scratch, cudaStream_t stream, std::string* err) {
    int32_t* valid = static_cast<int32_t*>(scratch);
    Entry* sorted = reinterpret_cast<Entry*>(static_cast<char*>(scratch) + 16);
    float* parts = reinterpret_cast<float*>(sorted + (M + 1) / 2 * 2);
    launch_pdl(sort_tokens_kernel, dim3((unsigned)((v + BINS - 1) / BINS)), dim3(SORT_WARPS * 32), 0, stream, ids,
               static_cast<long long>(M), static_cast<int>(v), sorted, valid, h, accumulate ? nullptr : dE);
    int rc = check("token sort kernel", err);
    if (rc || M == 0) return rc;
    const int part = part_tokens(M, h), nv = h / 8, threads = std::min(SUM_THREADS, (nv + 31) / 32 * 32);
    const dim3 grid((unsigned)((M + part - 1) / part), (unsigned)((nv + threads - 1) / threads));
    launch_pdl(embedding_sum_kernel, grid, dim3(threads), 0, stream, static_cast<const Entry*>(sorted),
               static_cast<const int32_t*>(valid), part, h, scale, static_cast<const __nv_bfloat16*>(dOut), dE, accumulate,
               parts);
    if ((rc = check("embedding gradient kernel", err)) || grid.x == 1) return rc;
    launch_pdl(embedding_join_kernel, grid, dim3(threads), 0, stream, static_cast<const Entry*>(sorted),
               static_cast<const int32_t*>(valid), part, h, scale, dE, accumulate, static_cast<const float*>(parts));
    return check("embedding join kernel", err);
}

int vocab_loss_launch(const void* logits, int64_t M, int64_t v, const int32_t* labels, const float* dloss, float* loss,
                      void* dlogits, cudaStream_t stream, std::string* err) {
    if (M == 0) return TP_OK;
    launch_pdl(loss_kernel, dim3((unsigned)M), dim3(LOSS_THREADS), 0, stream, static_cast<const __nv_bfloat16*>(logits),
               static_cast<int>(v), labels, dloss, loss, static_cast<__nv_bfloat16*>(dlogits));
    return check("loss kernel", err);
}

}  // namespace tpi
