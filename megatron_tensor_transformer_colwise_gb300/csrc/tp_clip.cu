// tp_clip.cu -- the norm of all gradients together, and clipping by it:
//   N = sqrt(sum over all tensors and elements of g^2),
//   dst = g min(1, max_norm / N).
//
// Two passes over the data, since no element can be scaled before all are
// summed: one kernel leaves a sum a CTA, the other adds these sums in a fixed
// order (in every CTA, the same bits) and scales.  The tensors' addresses and
// sizes travel in the kernels' parameters, so nothing is copied to the device
// before a call and a captured call is complete by itself.
//
// Both passes are bound by memory: 218 million fp32 gradients 395 us, where reading
// them twice and writing them once takes 386 at the copy rate (the sum alone 6.1
// TB/s, the second pass 6.6); 8.4 million 18.4 us, where the second pass reads from
// L2, of which two launches and the sums' way from one to the other are about 8.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <float.h>

#include <algorithm>
#include <string>

#include "tp_device.cuh"
#include "tp_internal.h"

namespace {

using namespace tpk;

constexpr int THREADS = 256, CTAS = 4;  // CTAs an SM
constexpr int CHUNK = 8192;       // elements that a CTA takes at a time
// Chunks at the end (half of L2) that the sums leave there for the second pass, all
// others giving way first: 218 million gradients 395 us, 400 without, 398 with half
// as many.
constexpr int KEEP = 2000;
constexpr int MAX_GRID = 2048;    // CTAs of a launch, and the sums kept for it
constexpr int FEW = 32, MANY = 512;  // tensors of a launch

struct Tensor {
    const void* src;
    void* dst;
    long long n, first;  // elements; first chunk
    int bf16;
};
template <int CAP>
struct Tensors {
    Tensor t[CAP];
    int count;
    long long chunks;
};

template <int CAP>
__device__ __forceinline__ const Tensor& tensor_of(const Tensors<CAP>& p, long long chunk) {
    int lo = 0, hi = p.count - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (p.t[mid].first <= chunk) lo = mid;
        else hi = mid - 1;
    }
    return p.t[lo];
}

// A chunk is PIECES 16-byte pieces a thread of fp32, half as many of bf16, all
// read before the first is used: 32 KB in flight a CTA.
constexpr int PIECES = CHUNK / 4 / THREADS;

template <bool BF16>
__device__ __forceinline__ void unpack(const uint4& u, float (&f)[BF16 ? 8 : 4]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (BF16) {
            const float2 p = unpack_bf16x2(w[i]);
            f[(2 * i) % (BF16 ? 8 : 4)] = p.x;
            f[(2 * i + 1) % (BF16 ? 8 : 4)] = p.y;
        } else {
            f[i] = __uint_as_float(w[i]);
        }
    }
}

template <bool BF16>
__device__ __forceinline__ float value_at(const void* src, long long i) {
    return BF16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(src)[i]) : static_cast<const float*>(src)[i];
}

template <bool BF16>
__device__ __forceinline__ void store_at(void* dst, long long i, float g) {
    if (BF16) static_cast<__nv_bfloat16*>(dst)[i] = __float2bfloat16_rn(g);
    else static_cast<float*>(dst)[i] = g;
}

// Calls one(i) for this thread's elements [from, to) of a tensor that are not
// in a whole 16-byte piece: the last chunk's last few.
template <int N, typename F>
__device__ __forceinline__ void for_rest(long long from, long long to, F&& one) {
    const long long i = from + (to - from) / N * N + threadIdx.x;
    if (threadIdx.x < N && i < to) one(i);
}

// A sum as a number and what its roundings left (two-sum: exact but for the
// roundings of lo), since 64-bit arithmetic is 64 times slower here: with doubles
// in every thread the two launches spent 15 of 25 us on a GeLU MLP's gradients in
// them.
struct Sum {
    float hi = 0.0f, lo = 0.0f;
    __device__ __forceinline__ void add(float t) {
        const float s = hi + t, b = s - hi;
        lo += (hi - (s - b)) + (t - b);
        hi = s;
    }
};

// Adds this thread's part of a chunk's sum of squares to sum, or, where it is out
// of sum's range, to far.
template <bool BF16>
__device__ __forceinline__ void chunk_sum(const void* src, long long from, long long to, bool keep, Sum& sum, double& far) {
    constexpr int N = BF16 ? 8 : 4, P = BF16 ? PIECES / 2 : PIECES;
    const uint4* at = reinterpret_cast<const uint4*>(static_cast<const char*>(src) + from * (16 / N));
    const int pieces = static_cast<int>((to - from) / N);
    uint4 u[P];
#pragma unroll
    for (int k = 0; k < P; ++k) {
        const int v = threadIdx.x + k * THREADS;
        u[k] = v < pieces ? (keep ? at[v] : __ldcs(at + v)) : make_uint4(0u, 0u, 0u, 0u);
    }
    float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    uint32_t any = 0;
#pragma unroll
    for (int k = 0; k < P; ++k) {
        float f[N];
        unpack<BF16>(u[k], f);
#pragma unroll
        for (int e = 0; e < N; ++e) s[e & 3] = fmaf(f[e], f[e], s[e & 3]);
        any |= u[k].x | u[k].y | u[k].z | u[k].w;
    }
    float t = (s[0] + s[1]) + (s[2] + s[3]);
    for_rest<N>(from, to, [&](long long i) {
        const float g = value_at<BF16>(src, i);
        t = fmaf(g, g, t);
        any |= __float_as_uint(g);
    });
    // Squares near the ends of fp32's range are summed again in 64 bits: a sum
    // below 2^-90 may have lost some, and 2^18 chunks of 32 lanes stay finite below
    // 2^100.
    if (t >= 0x1p-90f && t <= 0x1p100f) {
        sum.add(t);
        return;
    }
    if (!(any & (BF16 ? 0x7fff7fffu : 0x7fffffffu))) return;  // zeros of either sign
    double d = 0.0;
#pragma unroll 1
    for (int v = threadIdx.x; v < pieces; v += THREADS) {
        float f[N];
        unpack<BF16>(at[v], f);
#pragma unroll
        for (int e = 0; e < N; ++e) d = fma(static_cast<double>(f[e]), static_cast<double>(f[e]), d);
    }
    for_rest<N>(from, to, [&](long long i) {
        const double g = value_at<BF16>(src, i);
        d = fma(g, g, d);
    });
    far += d;
}

template <int CAP>
__global__ void __launch_bounds__(THREADS, CTAS) grad_sum_kernel(const __grid_constant__ Tensors<CAP> p,
                                                                 double* sums) {
    constexpr int WARPS = THREADS / 32;
    __shared__ Sum red[WARPS];
    __shared__ double all[THREADS];
    pdl_trigger();
    pdl_wait();
    Sum sum;
    double far = 0.0;
    for (long long chunk = blockIdx.x; chunk < p.chunks; chunk += gridDim.x) {
        const Tensor& t = tensor_of(p, chunk);
        const long long from = (chunk - t.first) * CHUNK, to = min(from + CHUNK, t.n);
        const bool keep = chunk >= p.chunks - KEEP;
        if (t.bf16) chunk_sum<true>(t.src, from, to, keep, sum, far);
        else chunk_sum<false>(t.src, from, to, keep, sum, far);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const float hi = __shfl_xor_sync(0xffffffffu, sum.hi, o), lo = __shfl_xor_sync(0xffffffffu, sum.lo, o);
        sum.add(hi);
        sum.lo += lo;
    }
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = sum;
    all[threadIdx.x] = far;
    const bool any_far = __syncthreads_or(far != 0.0);  // (true for NaN)
    if (threadIdx.x >= 32) return;
    double total = 0.0;
    if (threadIdx.x < WARPS) total = static_cast<double>(red[threadIdx.x].hi) + static_cast<double>(red[threadIdx.x].lo);
    for (int i = threadIdx.x; any_far && i < THREADS; i += 32) total += all[i];
#pragma unroll
    for (int o = any_far ? 16 : WARPS / 2; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
    if (threadIdx.x == 0) sums[blockIdx.x] = total;
}

// This thread's part of a chunk: dst = src times the factor.  Both sides are
// used once here, so neither stays in L2 ahead of what is still to be read.
template <bool BF16>
__device__ __forceinline__ void chunk_scale(const void* src, void* dst, long long from, long long to, double by) {
    constexpr int N = BF16 ? 8 : 4, P = BF16 ? PIECES / 2 : PIECES;
    const float factor = static_cast<float>(by);
    const uint4* at = reinterpret_cast<const uint4*>(static_cast<const char*>(src) + from * (16 / N));
    uint4* out = reinterpret_cast<uint4*>(static_cast<char*>(dst) + from * (16 / N));
    const int pieces = static_cast<int>((to - from) / N);
    uint4 u[P];
#pragma unroll
    for (int k = 0; k < P; ++k) {
        const int v = threadIdx.x + k * THREADS;
        if (v < pieces) u[k] = __ldcs(at + v);
    }
#pragma unroll
    for (int k = 0; k < P; ++k) {
        const int v = threadIdx.x + k * THREADS;
        if (v >= pieces) continue;
        float f[N];
        unpack<BF16>(u[k], f);
#pragma unroll
        for (int e = 0; e < N; ++e) f[e] *= factor;
        uint4 o;
        if (BF16)
            o = make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4 % N], f[5 % N]),
                           pack_bf16x2(f[6 % N], f[7 % N]));
        else
            o = make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
        __stcs(out + v, o);
    }
    for_rest<N>(from, to, [&](long long i) {
        store_at<BF16>(dst, i, value_at<BF16>(src, i) * factor);
    });
}

// The same where fp32 does not hold the factor in full (gradients near its
// largest number): in 64 bits, in code of its own.  With the choice made for
// each element, both products were computed: 1100 us for 218 million gradients.
template <bool BF16>
__device__ __noinline__ void chunk_scale_far(const void* src, void* dst, long long from, long long to, double by) {
#pragma unroll 1
    for (long long i = from + threadIdx.x; i < to; i += THREADS)
        store_at<BF16>(dst, i, static_cast<float>(value_at<BF16>(src, i) * by));
}

// 1 / sqrt(s) of a finite s > 0, by fp32's and one step of Newton's method (an
// error of 2^-22 becomes one of 2^-43); s is brought between 1 and 4 first, where
// fp32 holds it.
__device__ __forceinline__ double inverse_root(double s) {
    const int half = ((__double2hiint(s) >> 20) - 1023) >> 1;  // s is between 4^half and 4^(half + 1)
    const double m = __hiloint2double(__double2hiint(s) - half * (1 << 21), __double2loint(s));
    const double y = rsqrtf(static_cast<float>(m)), z = y * (1.5 - 0.5 * m * y * y);
    return z * __hiloint2double((1023 - half) << 20, 0);
}

// n_sums: CTAs of all launches of grad_sum_kernel together.  The chunks run
// from the last to the first: the last ones that the sums read are in L2.
template <int CAP>
__global__ void __launch_bounds__(THREADS, CTAS) grad_scale_kernel(const __grid_constant__ Tensors<CAP> p,
                                                                   const double* sums, int n_sums,
                                                                   float max_norm, float* norm) {
    __shared__ double factor;
    pdl_trigger();
    pdl_wait();
    if (threadIdx.x < 32) {
        double s = 0.0;
        constexpr int LOADS = 20;  // a launch's sums at once, or nearly
        for (int i0 = threadIdx.x; i0 < n_sums; i0 += 32 * LOADS) {
            double v[LOADS];
#pragma unroll
            for (int k = 0; k < LOADS; ++k) v[k] = i0 + 32 * k < n_sums ? sums[i0 + 32 * k] : 0.0;
#pragma unroll
            for (int k = 0; k < LOADS; ++k) s += v[k];
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        if (threadIdx.x == 0) {
            // A norm that is not finite (an infinity or NaN among the gradients)
            // scales nothing; the caller sees it and skips the step.
            double length = s, by = 1.0;
            if (s > 0.0 && s <= DBL_MAX) {
                const double inverse = inverse_root(s);
                length = s * inverse;
                if (length > max_norm) by = fmin(1.0, max_norm * inverse);
            }
            if (norm && blockIdx.x == 0) *norm = static_cast<float>(length);
            factor = by;
        }
    }
    __syncthreads();
    const double by = factor;
    for (long long chunk = p.chunks - 1 - blockIdx.x; chunk >= 0; chunk -= gridDim.x) {
        const Tensor& t = tensor_of(p, chunk);
        if (!t.dst || (by == 1.0 && t.dst == t.src)) continue;
        const long long from = (chunk - t.first) * CHUNK, to = min(from + CHUNK, t.n);
        if (by < 0x1p-120) {
            if (t.bf16) chunk_scale_far<true>(t.src, t.dst, from, to, by);
            else chunk_scale_far<false>(t.src, t.dst, from, to, by);
        } else {
            if (t.bf16) chunk_scale<true>(t.src, t.dst, from, to, by);
            else chunk_scale<false>(t.src, t.dst, from, to, by);
        }
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

template <int CAP>
int fill(Tensors<CAP>& p, const tp_grad_tensor* g, int count) {
    p.count = count;
    long long at = 0;
    for (int i = 0; i < count; ++i) {
        p.t[i] = {g[i].src, g[i].dst, g[i].n, at, g[i].dtype == TP_BF16};
        at += (g[i].n + CHUNK - 1) / CHUNK;
    }
    p.chunks = at;
    return static_cast<int>(std::max(1LL, std::min<long long>({at, tpi::device_sm_count() * static_cast<long long>(CTAS), MAX_GRID})));
}

template <int CAP>
int launch(const tp_grad_tensor* g, int count, float max_norm, float* norm, double* sums, cudaStream_t stream,
           std::string* err) {
    Tensors<CAP> p;
    int n_sums = 0;
    for (int at = 0; at < count || at == 0; at += CAP) {
        const int grid = fill(p, g + at, std::min(CAP, count - at));
        tpi::launch_pdl(grad_sum_kernel<CAP>, dim3(grid), dim3(THREADS), 0, stream, p, sums + n_sums);
        const int rc = check("gradient norm kernel", err);
        if (rc) return rc;
        n_sums += grid;
    }
    for (int at = 0; at < count || at == 0; at += CAP) {
        const int grid = fill(p, g + at, std::min(CAP, count - at));
        tpi::launch_pdl(grad_scale_kernel<CAP>, dim3(grid), dim3(THREADS), 0, stream, p, static_cast<const double*>(sums),
                        n_sums, max_norm, at == 0 ? norm : nullptr);
        const int rc = check("gradient clipping kernel", err);
        if (rc) return rc;
    }
    return TP_OK;
}

}  // namespace

namespace tpi {

size_t grad_clip_scratch_bytes(int count) {
    return static_cast<size_t>(std::max(1, (count + MANY - 1) / MANY)) * MAX_GRID * sizeof(double);
}

int grad_clip_launch(const tp_grad_tensor* grads, int count, float max_norm, float* norm, void* scratch,
                     cudaStream_t stream, std::string* err) {
    double* sums = static_cast<double*>(scratch);
    return count <= FEW ? launch<FEW>(grads, count, max_norm, norm, sums, stream, err)
                        : launch<MANY>(grads, count, max_norm, norm, sums, stream, err);
}

}  // namespace tpi
