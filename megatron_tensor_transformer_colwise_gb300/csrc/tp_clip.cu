// tp_clip.cu -- the norm of all gradients together, and clipping by it:
//   N = sqrt(sum over all tensors and elements of g^2),
//   dst = g min(1, max_norm / N).
//
// Two passes over the data, since no element can be scaled before all are
// summed: one kernel leaves a sum a CTA, the other adds these sums in a fixed
// order (in every CTA, the same bits) and scales.  The tensors' addresses and
// sizes travel in the kernels' parameters, so nothing is copied to the device
// before a call and a captured call is complete by itself.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <float.h>

#include <algorithm>
#include <string>

#include "tp_device.cuh"
#include "tp_internal.h"

namespace {

using namespace tpk;

constexpr int THREADS = 256;
constexpr int CHUNK = 8192;       // elements that a CTA takes at a time
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

__device__ __forceinline__ float value_at(const Tensor& t, long long i) {
    return t.bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(t.src)[i]) : static_cast<const float*>(t.src)[i];
}

template <int CAP>
__global__ void __launch_bounds__(THREADS) grad_sum_kernel(const __grid_constant__ Tensors<CAP> p, double* __restrict__ sums) {
    __shared__ double red[THREADS / 32];
    pdl_trigger();
    pdl_wait();
    double total = 0.0;
    for (long long chunk = blockIdx.x; chunk < p.chunks; chunk += gridDim.x) {
        const Tensor& t = tensor_of(p, chunk);
        const long long from = (chunk - t.first) * CHUNK, to = min(from + CHUNK, t.n);
        float s = 0.0f;
        unsigned any = 0;
        for (long long i = from + threadIdx.x; i < to; i += THREADS) {
            const float g = value_at(t, i);
            s = fmaf(g, g, s);
            any |= __float_as_uint(g) << 1;
        }
        // Squares that leave fp32's range (a sum below 2^-90 may have lost
        // some, one above the largest number has) are summed again in 64 bits.
        if (any && !(s >= 0x1p-90f && s <= FLT_MAX)) {
            double d = 0.0;
            for (long long i = from + threadIdx.x; i < to; i += THREADS) {
                const double g = value_at(t, i);
                d = fma(g, g, d);
            }
            total += d;
        } else {
            total += s;
        }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = total;
    __syncthreads();
    if (threadIdx.x == 0) {
        total = 0.0;
        for (int w = 0; w < THREADS / 32; ++w) total += red[w];
        sums[blockIdx.x] = total;
    }
}

// n_sums: CTAs of all launches of grad_sum_kernel together.
template <int CAP>
__global__ void __launch_bounds__(THREADS) grad_scale_kernel(const __grid_constant__ Tensors<CAP> p,
                                                             const double* __restrict__ sums, int n_sums, float max_norm,
                                                             float* norm) {
    __shared__ double red[THREADS / 32];
    pdl_trigger();
    pdl_wait();
    double s = 0.0;
    for (int i = threadIdx.x; i < n_sums; i += THREADS) s += sums[i];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = s;
    __syncthreads();
    s = 0.0;
    for (int w = 0; w < THREADS / 32; ++w) s += red[w];
    const double length = sqrt(s);
    if (norm && blockIdx.x == 0 && threadIdx.x == 0) *norm = static_cast<float>(length);
    // A norm that is not finite (an infinity or NaN among the gradients)
    // scales nothing; the caller sees it and skips the step.
    double by = 1.0;
    if (length > max_norm && length <= DBL_MAX) by = max_norm / length;
    // A factor that fp32 does not hold in full (gradients near its largest
    // number) multiplies in 64 bits.
    const bool tiny = by < 0x1p-120;
    const float factor = static_cast<float>(by);
    for (long long chunk = blockIdx.x; chunk < p.chunks; chunk += gridDim.x) {
        const Tensor& t = tensor_of(p, chunk);
        if (!t.dst || (by == 1.0 && t.dst == t.src)) continue;
        const long long from = (chunk - t.first) * CHUNK, to = min(from + CHUNK, t.n);
        for (long long i = from + threadIdx.x; i < to; i += THREADS) {
            const float v = value_at(t, i), g = tiny ? static_cast<float>(v * by) : v * factor;
            if (t.bf16) static_cast<__nv_bfloat16*>(t.dst)[i] = __float2bfloat16_rn(g);
            else static_cast<float*>(t.dst)[i] = g;
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
    return static_cast<int>(std::max(1LL, std::min<long long>({at, tpi::device_sm_count() * 8LL, MAX_GRID})));
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
