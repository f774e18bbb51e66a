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

// Tokens sorted by word.  A CTA owns BINS words and looks through all ids: it
// counts the tokens of words below its own (its place in the order) and of
// each of its own, then puts the positions down word by word.  Every warp
// takes a contiguous part of the tokens and has counters of its own, so the
// positions of a word come out ascending whatever the order of the work.
//   order: positions by word; start[r] .. start[r + 1]: those of word r.
constexpr int BINS = 256, SORT_WARPS = 32;

__global__ void __launch_bounds__(SORT_WARPS * 32) sort_tokens_kernel(const int32_t* __restrict__ ids, int M, int v,
                                                                     int32_t* __restrict__ order, int32_t* __restrict__ start) {
    __shared__ int32_t count[SORT_WARPS][BINS];
    __shared__ int32_t below[SORT_WARPS], sums[BINS / 32];
    pdl_trigger();
    pdl_wait();
    const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int lo = blockIdx.x * BINS, bins = min(BINS, v - lo);
    for (int b = lane; b < BINS; b += 32) count[w][b] = 0;
    __syncwarp();
    const int part = ((M + SORT_WARPS - 1) / SORT_WARPS + 31) / 32 * 32;
    const long long from = static_cast<long long>(w) * part, to = min(from + part, static_cast<long long>(M));
    int under = 0;
    for (long long i = from + lane; i < to; i += 32) {
        const int id = ids[i];
        under += id >= 0 && id < lo;
        if (id >= lo && id - lo < bins) atomicAdd(&count[w][id - lo], 1);
    }
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
        if (threadIdx.x < bins) start[lo + threadIdx.x] = base;
        if (lo + static_cast<int>(threadIdx.x) == v - 1) start[v] = base + total;
    }
    __syncthreads();
    for (long long at = from; at < to; at += 32) {
        const long long i = at + lane;
        const int id = i < to ? ids[i] : -1;
        const bool mine = id >= lo && id - lo < bins;
        const unsigned live = __ballot_sync(0xffffffffu, mine);
        if (mine) {
            const int b = id - lo;
            const unsigned same = __match_any_sync(live, b);
            const unsigned before = same & ((1u << lane) - 1u);
            const int place = count[w][b] + __popc(before);
            order[place] = static_cast<int32_t>(i);
            __syncwarp(live);
            if (!before) count[w][b] += __popc(same);
        }
        __syncwarp();
    }
}

// One CTA per word: dE[r] (+)= scale * sum of its tokens' rows, in order.
constexpr int SUM_THREADS = 128;

__global__ void __launch_bounds__(SUM_THREADS) embedding_sum_kernel(const int32_t* __restrict__ order,
                                                                   const int32_t* __restrict__ start, int h, float scale,
                                                                   const __nv_bfloat16* __restrict__ dOut, float* dE,
                                                                   int accumulate) {
    pdl_trigger();
    pdl_wait();
    const long long r = blockIdx.x;
    const int from = start[r], to = start[r + 1];
    if (accumulate && from == to) return;
    for (int c = threadIdx.x; c < h >> 3; c += SUM_THREADS) {
        float s[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f}, f[8];
        for (int k = from; k < to; ++k) {
            unpack8(reinterpret_cast<const uint4*>(dOut + static_cast<long long>(order[k]) * h)[c], f);
#pragma unroll
            for (int e = 0; e < 8; ++e) s[e] += f[e];
        }
        float4* out = reinterpret_cast<float4*>(dE + r * h) + 2 * c;
        float4 a = make_float4(0, 0, 0, 0), b = a;
        if (accumulate) {
            a = out[0];
            b = out[1];
        }
        out[0] = make_float4(fmaf(scale, s[0], a.x), fmaf(scale, s[1], a.y), fmaf(scale, s[2], a.z), fmaf(scale, s[3], a.w));
        out[1] = make_float4(fmaf(scale, s[4], b.x), fmaf(scale, s[5], b.y), fmaf(scale, s[6], b.z), fmaf(scale, s[7], b.w));
    }
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

size_t vocab_embedding_bwd_scratch_bytes(int64_t M, int64_t v, int h) {
    return static_cast<size_t>((v + 1 + 3) / 4 * 4 + M) * sizeof(int32_t);
}

int vocab_embedding_bwd_launch(const int32_t* ids, int64_t M, int64_t v, int h, float scale, const void* dOut, float* dE,
                               int accumulate, void* scratch, cudaStream_t stream, std::string* err) {
    int32_t* start = static_cast<int32_t*>(scratch);
    int32_t* order = start + (v + 1 + 3) / 4 * 4;
    launch_pdl(sort_tokens_kernel, dim3((unsigned)((v + BINS - 1) / BINS)), dim3(SORT_WARPS * 32), 0, stream, ids,
               static_cast<int>(M), static_cast<int>(v), order, start);
    int rc = check("token sort kernel", err);
    if (rc) return rc;
    launch_pdl(embedding_sum_kernel, dim3((unsigned)v), dim3(SUM_THREADS), 0, stream, static_cast<const int32_t*>(order),
               static_cast<const int32_t*>(start), h, scale, static_cast<const __nv_bfloat16*>(dOut), dE, accumulate);
    return check("embedding gradient kernel", err);
}

int vocab_loss_launch(const void* logits, int64_t M, int64_t v, const int32_t* labels, const float* dloss, float* loss,
                      void* dlogits, cudaStream_t stream, std::string* err) {
    if (M == 0) return TP_OK;
    launch_pdl(loss_kernel, dim3((unsigned)M), dim3(LOSS_THREADS), 0, stream, static_cast<const __nv_bfloat16*>(logits),
               static_cast<int>(v), labels, dloss, loss, static_cast<__nv_bfloat16*>(dlogits));
    return check("loss kernel", err);
}

}  // namespace tpi
