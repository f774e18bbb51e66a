// tp_layernorm.cu -- layer norm with a gain and a bias, and its gradients.
//
// Source: "텐서 병렬화" (itwiki, Tensor parallelism), section "통신 연산 f와
// g": norms are replicated, so every shard's norm is this one.  With
// mu = mean_j x_j, r = 1 / sqrt(mean_j (x_j - mu)^2 + eps), xh = (x - mu) r:
//   y      = xh gain + bias
//   dx     = dres + r (g - mean_j g_j - xh mean_j g_j xh_j),   g = dy gain
//   dgain  = sum over rows of dy xh,   dbias = sum over rows of dy
//
// Both directions are bound by memory.  A row stays in the registers of W
// warps (VPT 16-byte pieces a thread), so each input is read once and each
// output written once; a CTA of THREADS holds THREADS / (32 W) rows at a time
// and strides over the rows, with the gain and the bias kept in registers.
// The weights' gradients are summed in registers over a CTA's rows, and a
// second kernel adds the CTAs' sums in a fixed order: no atomics, so repeated
// calls give the same bits.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <string>
#include <type_traits>

#include "tp_device.cuh"
#include "tp_internal.h"

namespace {

using namespace tpk;

constexpr int THREADS = 512;
constexpr int MAX_PARTS = 512;  // most CTAs of the gradients' kernel

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

__device__ __forceinline__ uint4 zeros8() { return make_uint4(0u, 0u, 0u, 0u); }
__device__ __forceinline__ uint4 ones8() { return make_uint4(0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u); }

// Sums of N values over the W warps of a row.  `red` holds two slots of W
// values for each of N, used in turn, so that one barrier a sum is enough.
template <int W, int N>
struct RowSum {
    float* red;
    int turn = 0;
    __device__ __forceinline__ explicit RowSum(float* r) : red(r) {}
    __device__ __forceinline__ void operator()(float (&v)[N]) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
        }
        if (W == 1) return;
        const int group = threadIdx.x / (32 * W), w = threadIdx.x / 32 % W;
        float* at = red + (group * 2 + turn) * N * W;
        if ((threadIdx.x & 31) == 0) {
#pragma unroll
            for (int i = 0; i < N; ++i) at[i * W + w] = v[i];
        }
        named_bar_sync(1 + group, 32 * W);
#pragma unroll
        for (int i = 0; i < N; ++i) {
            v[i] = 0.0f;
#pragma unroll
            for (int k = 0; k < W; ++k) v[i] += at[i * W + k];
        }
        turn ^= 1;
    }
};

// Mean and 1 / sqrt(variance + eps) of a row in registers: the mean first, so
// that a row whose mean is far from zero keeps its variance.
template <int W, int VPT>
__device__ __forceinline__ float2 row_stats(const float (&f)[VPT][8], int first, int nv, float inv_h, float eps,
                                            RowSum<W, 1>& sum) {
    float s[1] = {0.0f};
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
#pragma unroll
        for (int e = 0; e < 8; ++e) s[0] += f[i][e];  // pieces past the row hold zeros
    }
    sum(s);
    const float mean = s[0] * inv_h;
    s[0] = 0.0f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        if (first + i * 32 * W >= nv) continue;
#pragma unroll
        for (int e = 0; e < 8; ++e) s[0] = fmaf(f[i][e] - mean, f[i][e] - mean, s[0]);
    }
    sum(s);
    return make_float2(mean, rsqrtf(s[0] * inv_h + eps));
}

template <int W, int VPT>
__global__ void __launch_bounds__(THREADS) layernorm_kernel(const __nv_bfloat16* x, long long rows, int h,
                                                            const __nv_bfloat16* __restrict__ gain,
                                                            const __nv_bfloat16* __restrict__ bias, float eps,
                                                            __nv_bfloat16* y, float* __restrict__ stats) {
    constexpr int GROUPS = THREADS / (32 * W);
    __shared__ float red[GROUPS * 2 * W];
    pdl_trigger();
    pdl_wait();
    RowSum<W, 1> sum(red);
    const int first = threadIdx.x % (32 * W), nv = h >> 3;
    const float inv_h = 1.0f / static_cast<float>(h);
    uint4 gv[VPT], bv[VPT];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int v = first + i * 32 * W;
        gv[i] = gain && v < nv ? reinterpret_cast<const uint4*>(gain)[v] : ones8();
        bv[i] = bias && v < nv ? reinterpret_cast<const uint4*>(bias)[v] : zeros8();
    }
    for (long long row = static_cast<long long>(blockIdx.x) * GROUPS + threadIdx.x / (32 * W); row < rows;
         row += static_cast<long long>(gridDim.x) * GROUPS) {
        float f[VPT][8];
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int v = first + i * 32 * W;
            unpack8(v < nv ? reinterpret_cast<const uint4*>(x + row * h)[v] : zeros8(), f[i]);
        }
        const float2 st = row_stats<W, VPT>(f, first, nv, inv_h, eps, sum);
        if (stats && first == 0) {
            stats[row] = st.x;
            stats[rows + row] = st.y;
        }
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int v = first + i * 32 * W;
            if (v >= nv) continue;
            float g[8], b[8];
            unpack8(gv[i], g);
            unpack8(bv[i], b);
#pragma unroll
            for (int e = 0; e < 8; ++e) f[i][e] = fmaf((f[i][e] - st.x) * st.y, g[e], b[e]);
            reinterpret_cast<uint4*>(y + row * h)[v] = pack8(f[i]);
        }
    }
}

// dx of every row, and the CTA's sums for dgain and dbias in parts
// [CTAs][2][h].  dx may be dy or dres: a row's inputs are in registers before
// its outputs are stored, and no other row's are touched.
template <int W, int VPT>
__global__ void __launch_bounds__(THREADS) layernorm_bwd_kernel(const __nv_bfloat16* __restrict__ x, long long rows, int h,
                                                                const __nv_bfloat16* __restrict__ gain, float eps,
                                                                const float* __restrict__ stats, const __nv_bfloat16* dy,
                                                                const __nv_bfloat16* dres, __nv_bfloat16* dx,
                                                                float* __restrict__ parts) {
    constexpr int GROUPS = THREADS / (32 * W);
    __shared__ float red[GROUPS * 2 * W * 3];
    pdl_trigger();
    pdl_wait();
    RowSum<W, 1> sum(red);
    RowSum<W, 2> sums(red + GROUPS * 2 * W);
    const int first = threadIdx.x % (32 * W), nv = h >> 3, group = threadIdx.x / (32 * W);
    const float inv_h = 1.0f / static_cast<float>(h);
    uint4 gv[VPT];
    float dg[VPT][8], db[VPT][8];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int v = first + i * 32 * W;
        gv[i] = gain && v < nv ? reinterpret_cast<const uint4*>(gain)[v] : ones8();
#pragma unroll
        for (int e = 0; e < 8; ++e) dg[i][e] = db[i][e] = 0.0f;
    }
    for (long long row = static_cast<long long>(blockIdx.x) * GROUPS + group; row < rows;
         row += static_cast<long long>(gridDim.x) * GROUPS) {
        float f[VPT][8];
        uint4 dv[VPT];
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int v = first + i * 32 * W;
            unpack8(v < nv ? reinterpret_cast<const uint4*>(x + row * h)[v] : zeros8(), f[i]);
            dv[i] = v < nv ? reinterpret_cast<const uint4*>(dy + row * h)[v] : zeros8();
        }
        const float2 st = stats ? make_float2(stats[row], stats[rows + row])
                                : row_stats<W, VPT>(f, first, nv, inv_h, eps, sum);
        float s[2] = {0.0f, 0.0f};
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            float g[8], d[8];
            unpack8(gv[i], g);
            unpack8(dv[i], d);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                f[i][e] = (f[i][e] - st.x) * st.y;
                dg[i][e] = fmaf(d[e], f[i][e], dg[i][e]);
                db[i][e] += d[e];
                s[0] = fmaf(d[e], g[e], s[0]);
                s[1] = fmaf(d[e] * g[e], f[i][e], s[1]);
            }
        }
        sums(s);
        const float c1 = s[0] * inv_h, c2 = s[1] * inv_h;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int v = first + i * 32 * W;
            if (v >= nv) continue;
            float g[8], d[8], a[8];
            unpack8(gv[i], g);
            unpack8(dv[i], d);
            unpack8(dres ? reinterpret_cast<const uint4*>(dres + row * h)[v] : zeros8(), a);
#pragma unroll
            for (int e = 0; e < 8; ++e) a[e] = fmaf(st.y, fmaf(-f[i][e], c2, fmaf(d[e], g[e], -c1)), a[e]);
            reinterpret_cast<uint4*>(dx + row * h)[v] = pack8(a);
        }
    }
    if (!parts) return;
    // The CTA's rows at a time are added in shared memory, group by group.
    extern __shared__ float cols[];  // [2][h] where GROUPS > 1
    float* out = parts + static_cast<long long>(blockIdx.x) * 2 * h;
    for (int k = 0; k < GROUPS; ++k) {
        if (k == group) {
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                const int v = first + i * 32 * W;
                if (v >= nv) continue;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const int c = v * 8 + e;
                    if (k) {
                        dg[i][e] += cols[c];
                        db[i][e] += cols[h + c];
                    }
                    if (k + 1 < GROUPS) {
                        cols[c] = dg[i][e];
                        cols[h + c] = db[i][e];
                    } else {
                        out[c] = dg[i][e];
                        out[h + c] = db[i][e];
                    }
                }
            }
        }
        if (GROUPS > 1) __syncthreads();
    }
}

// dgain (+)= and dbias (+)= the CTAs' sums, in order: 32 columns a CTA, eight
// warps that take every eighth part, joined in order.
constexpr int JOIN_WARPS = 8;

__global__ void __launch_bounds__(JOIN_WARPS * 32) layernorm_join_kernel(const float* __restrict__ parts, int n, int h,
                                                                        float* dgain, float* dbias, int accumulate) {
    pdl_trigger();
    pdl_wait();
    __shared__ float sum[JOIN_WARPS][32];
    float* out = blockIdx.y ? dbias : dgain;
    if (!out) return;
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
    float s = 0.0f;
    if (c < h) {
        for (int k = w; k < n; k += JOIN_WARPS) s += parts[(static_cast<long long>(k) * 2 + blockIdx.y) * h + c];
    }
    sum[w][lane] = s;
    __syncthreads();
    if (w || c >= h) return;
    s = 0.0f;
#pragma unroll
    for (int k = 0; k < JOIN_WARPS; ++k) s += sum[k][lane];
    out[c] = accumulate ? out[c] + s : s;
}

int check(const char* what, std::string* err) {
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) {
        if (err) *err = std::string(what) + ": " + cudaGetErrorString(e);
        return TP_ERR_CUDA;
    }
    return TP_OK;
}

template <int N>
using Int = std::integral_constant<int, N>;

// Warps of a row and 16-byte pieces a thread for rows of h: one warp up to
// 512 columns (no barrier), two pieces a thread up to 8192, then four.
template <typename F>
int for_width(int h, F&& f) {
    const int nv = h / 8;
    if (nv <= 32) return f(Int<1>(), Int<1>());
    if (nv <= 64) return f(Int<1>(), Int<2>());
    if (nv <= 128) return f(Int<2>(), Int<2>());
    if (nv <= 256) return f(Int<4>(), Int<2>());
    if (nv <= 512) return f(Int<8>(), Int<2>());
    if (nv <= 1024) return f(Int<16>(), Int<2>());
    return f(Int<16>(), Int<4>());
}

}  // namespace

namespace tpi {

int layernorm_launch(const void* x, int64_t rows, int h, const void* gain, const void* bias, float eps, void* y,
                     float* stats, cudaStream_t stream, std::string* err) {
    if (rows == 0) return TP_OK;
    return for_width(h, [&](auto W, auto VPT) {
        constexpr int GROUPS = THREADS / (32 * decltype(W)::value);
        const int64_t grid = std::min<int64_t>((rows + GROUPS - 1) / GROUPS, device_sm_count() * 4);
        launch_pdl(layernorm_kernel<decltype(W)::value, decltype(VPT)::value>, dim3((unsigned)grid), dim3(THREADS), 0,
                   stream, static_cast<const __nv_bfloat16*>(x), static_cast<long long>(rows), h,
                   static_cast<const __nv_bfloat16*>(gain), static_cast<const __nv_bfloat16*>(bias), eps,
                   static_cast<__nv_bfloat16*>(y), stats);
        return check("layer norm kernel", err);
    });
}

size_t layernorm_bwd_scratch_bytes(int64_t rows, int h) {
    return static_cast<size_t>(std::min<int64_t>(rows, MAX_PARTS)) * 2 * h * sizeof(float);
}

int layernorm_bwd_launch(const void* x, int64_t rows, int h, const void* gain, float eps, const float* stats,
                         const void* dy, const void* dres, void* dx, float* dgain, float* dbias, int accumulate,
                         void* scratch, cudaStream_t stream, std::string* err) {
    int64_t grid = 0;
    const bool weights = dgain || dbias;
    if (rows > 0) {
        const int rc = for_width(h, [&](auto W, auto VPT) {
            constexpr int GROUPS = THREADS / (32 * decltype(W)::value);
            auto kern = layernorm_bwd_kernel<decltype(W)::value, decltype(VPT)::value>;
            grid = std::min<int64_t>({(rows + GROUPS - 1) / GROUPS, device_sm_count(), MAX_PARTS});
            const size_t smem = GROUPS > 1 && weights ? static_cast<size_t>(h) * 2 * sizeof(float) : 0;
            launch_pdl(kern, dim3((unsigned)grid), dim3(THREADS), smem, stream, static_cast<const __nv_bfloat16*>(x),
                       static_cast<long long>(rows), h, static_cast<const __nv_bfloat16*>(gain), eps, stats,
                       static_cast<const __nv_bfloat16*>(dy), static_cast<const __nv_bfloat16*>(dres),
                       static_cast<__nv_bfloat16*>(dx), weights ? static_cast<float*>(scratch) : nullptr);
            return check("layer norm gradient kernel", err);
        });
        if (rc) return rc;
    }
    if (!weights) return TP_OK;
    launch_pdl(layernorm_join_kernel, dim3((h + 31) / 32, 2), dim3(JOIN_WARPS * 32), 0, stream,
               static_cast<const float*>(scratch), static_cast<int>(grid), h, dgain, dbias, accumulate);
    return check("layer norm join kernel", err);
}

}  // namespace tpi
