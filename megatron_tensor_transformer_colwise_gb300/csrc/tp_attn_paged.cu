// tp_attn_paged.cu -- causal GQA attention of new tokens over a paged
// key/value cache.
//
// For query head j of a token at position p, with KV head g = j / (a/k):
//   O = sum_{p' <= p} e^{s_p' - m} V[p'] / sum_{p' <= p} e^{s_p' - m},
//   s_p' = Q . K[p'] / sqrt d,   m the running maximum,
// one pass over the keys, fp32 throughout.
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <string>

#include "tp_device.cuh"
#include "tp_internal.h"
#include "tp_paged.cuh"

namespace {

using namespace tpk;

struct PagedAttnParams {
    PagedView v;
    const void *K, *V;
    const float *k_scale, *v_scale;
    const __nv_bfloat16* qkv;
    long long ld_qkv;
    __nv_bfloat16* o;
    int heads, heads_per_shard, shard_w, group;
    float scale_log2;
    int zero_rest;
    unsigned* status;
};

template <int D, bool E4M3>
__device__ __forceinline__ void load_row(const void* base, const float* scale, long long at, int lane,
                                         float (&x)[D / 32]) {
    if constexpr (E4M3) {
        const uint8_t* r = static_cast<const uint8_t*>(base) + at * D;
#pragma unroll
        for (int e = 0; e < D / 32; ++e)
            x[e] = __half2float(__half(__nv_cvt_fp8_to_halfraw(r[e * 32 + lane], __NV_E4M3))) * scale[at];
    } else {
        const __nv_bfloat16* r = static_cast<const __nv_bfloat16*>(base) + at * D;
#pragma unroll
        for (int e = 0; e < D / 32; ++e) x[e] = __bfloat162float(r[e * 32 + lane]);
    }
}

// One warp per (new token, query head); a key at a time, lanes over d.
template <int D, bool E4M3>
__global__ void __launch_bounds__(256) attn_paged_simple_kernel(const PagedAttnParams p) {
    pdl_trigger();
    pdl_wait();
    const int lane = threadIdx.x & 31;
    const long long n_items = p.v.rows * p.heads;
    const long long warps = static_cast<long long>(gridDim.x) * 8;
    for (long long it = static_cast<long long>(blockIdx.x) * 8 + (threadIdx.x >> 5); it < n_items; it += warps) {
        const int j = static_cast<int>(it % p.heads);
        const long long row = it / p.heads;
        __nv_bfloat16* o = p.o + row * p.heads * D + j * D;
        const int s = paged_owner(p.v, row);
        if (s < 0) {
            if (p.zero_rest)
                for (int e = 0; e < D / 32; ++e) o[e * 32 + lane] = __float2bfloat16_rn(0.0f);
            continue;
        }
        const PagedSeq q = paged_seq(p.v, s);
        const int pos = q.len - q.n + static_cast<int>(row - q.row0);
        const __nv_bfloat16* x = p.qkv + row * p.ld_qkv + (j / p.heads_per_shard) * p.shard_w +
                                 (j % p.heads_per_shard) * D;
        float qv[D / 32], acc[D / 32], kv[D / 32];
#pragma unroll
        for (int e = 0; e < D / 32; ++e) {
            qv[e] = __bfloat162float(x[e * 32 + lane]);
            acc[e] = 0.0f;
        }
        float m = -INFINITY, l = 0.0f;
        for (int c = 0; c <= pos; ++c) {
            const long long page = paged_page(p.v, s, c);
            if (page < 0) {
                if (lane == 0 && p.status) atomicOr(p.status, kStatusPage);
            }
            const long long at = page < 0 ? 0 : paged_row(p.v, page, j / p.group, c);
            float dot = 0.0f;
            if (page >= 0) {
                load_row<D, E4M3>(p.K, p.k_scale, at, lane, kv);
#pragma unroll
                for (int e = 0; e < D / 32; ++e) dot += qv[e] * kv[e];
            }
            for (int f = 16; f > 0; f >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, f);
            dot *= p.scale_log2;
            const float nm = fmaxf(m, dot);
            const float alpha = exp2f(m - nm), w = exp2f(dot - nm);
            m = nm;
            l = l * alpha + w;
#pragma unroll
            for (int e = 0; e < D / 32; ++e) kv[e] = 0.0f;
            if (page >= 0) load_row<D, E4M3>(p.V, p.v_scale, at, lane, kv);
#pragma unroll
            for (int e = 0; e < D / 32; ++e) acc[e] = acc[e] * alpha + w * kv[e];
        }
        const float inv = l > 0.0f ? 1.0f / l : 0.0f;
#pragma unroll
        for (int e = 0; e < D / 32; ++e) o[e * 32 + lane] = __float2bfloat16_rn(acc[e] * inv);
    }
}

}  // namespace

namespace tpi {

size_t attn_paged_scratch_bytes(int head_dim) {
    (void)head_dim;
    return 0;
}

int attn_paged_launch(const PagedArgs& a, void* O, void* scratch, bool zero_rest, cudaStream_t stream,
                      std::string* err) {
    (void)scratch;
    PagedAttnParams p{};
    p.v = paged_view(a);
    p.K = a.K;
    p.V = a.V;
    p.k_scale = a.k_scale;
    p.v_scale = a.v_scale;
    p.qkv = static_cast<const __nv_bfloat16*>(a.QKV);
    p.ld_qkv = a.ld_qkv;
    p.o = static_cast<__nv_bfloat16*>(O);
    p.heads = a.heads;
    p.heads_per_shard = a.heads / a.t;
    p.shard_w = static_cast<int>(a.shard_w);
    p.group = a.heads / a.kv_heads;
    p.scale_log2 = 1.4426950408889634f / sqrtf(static_cast<float>(a.head_dim));
    p.zero_rest = zero_rest ? 1 : 0;
    p.status = a.status;
    const long long need = (a.tokens * a.heads + 7) / 8, most = static_cast<long long>(device_sm_count()) * 8;
    const dim3 grid(static_cast<unsigned>(need < most ? need : most)), block(256);
    cudaError_t e;
    if (a.head_dim == 128)
        e = a.e4m3 ? launch_pdl(attn_paged_simple_kernel<128, true>, grid, block, 0, stream, p)
                   : launch_pdl(attn_paged_simple_kernel<128, false>, grid, block, 0, stream, p);
    else
        e = a.e4m3 ? launch_pdl(attn_paged_simple_kernel<64, true>, grid, block, 0, stream, p)
                   : launch_pdl(attn_paged_simple_kernel<64, false>, grid, block, 0, stream, p);
    if (e == cudaSuccess) e = cudaGetLastError();
    if (e != cudaSuccess) {
        if (err) *err = std::string("paged attention launch: ") + cudaGetErrorString(e);
        return TP_ERR_CUDA;
    }
    return TP_OK;
}

}  // namespace tpi
