// tp_kv.cu -- the paged key/value cache: appending the new tokens' keys and
// values, as bf16 or quantised to 8 bits, and reading sequences back.
//
// Quantisation of one token and KV head, x[0..d): with amax = max |x_j| held
// to [2^-100, largest finite bf16],
//   scale = amax / 448,   code_j = e4m3(x_j (448 / amax)),   x_j ~ code_j scale.
// The lower end keeps 448 / amax finite and scale a normal number for rows of
// zeros and of the smallest values; the upper end gives an infinity the code
// 448.  The product with the rounded reciprocal is at most 448 (1 + 2^-23), so
// the saturating conversion never changes a finite value by more than its
// rounding.
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <string>

#include "tp_device.cuh"
#include "tp_internal.h"
#include "tp_paged.cuh"

namespace {

using namespace tpk;

constexpr float kE4M3Max = 448.0f;
constexpr float kAmaxFloor = 7.888609052210118e-31f;  // 2^-100
constexpr float kAmaxCeil = 3.3895313892515355e38f;   // largest finite bf16

struct KvParams {
    PagedView v;
    void *K, *V;
    float *k_scale, *v_scale;
    const __nv_bfloat16* qkv;
    long long ld_qkv;
    int shard_w, q_w, kv_w, kv_per_shard, t;
    unsigned* status;
    // read back
    __nv_bfloat16 *k_out, *v_out;
    long long max_len;
};

// One warp per (new token, KV head, K or V).
template <bool E4M3>
__global__ void __launch_bounds__(256) kv_write_kernel(const KvParams p) {
    pdl_trigger();
    pdl_wait();
    const int lane = threadIdx.x & 31;
    const int k = p.v.kv_heads, d = p.v.d;
    const long long n_items = p.v.rows * k * 2;
    const long long warps = static_cast<long long>(gridDim.x) * 8;
    for (long long it = static_cast<long long>(blockIdx.x) * 8 + (threadIdx.x >> 5); it < n_items; it += warps) {
        const bool is_v = it & 1;
        const int g = static_cast<int>((it >> 1) % k);
        const long long row = (it >> 1) / k;
        const int s = paged_owner(p.v, row);
        if (s < 0) continue;
        const PagedSeq q = paged_seq(p.v, s);
        const int pos = q.len - q.n + static_cast<int>(row - q.row0);
        const long long page = paged_page(p.v, s, pos);
        if (page < 0) {
            if (lane == 0 && pos >= 0 && p.status) atomicOr(p.status, kStatusPage);
            continue;
        }
        // k >= t: shard g / (k/t) holds g; k < t: shard g t / k is the first with a replica.
        const int shard = k >= p.t ? g / p.kv_per_shard : g * (p.t / k);
        const int local = k >= p.t ? g % p.kv_per_shard : 0;
        const __nv_bfloat16* x =
            p.qkv + row * p.ld_qkv + shard * p.shard_w + p.q_w + (is_v ? p.kv_w : 0) + local * d;
        const long long at = paged_row(p.v, page, g, pos);
        if constexpr (!E4M3) {
            __nv_bfloat16* y = static_cast<__nv_bfloat16*>(is_v ? p.V : p.K) + at * d;
            for (int c = lane; c < d; c += 32) y[c] = x[c];
        } else {
            float amax = 0.0f;
            for (int c = lane; c < d; c += 32) amax = fmaxf(amax, fabsf(__bfloat162float(x[c])));
            for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
            amax = fminf(fmaxf(amax, kAmaxFloor), kAmaxCeil);
            const float inv = __fdiv_rn(kE4M3Max, amax);
            uint8_t* y = static_cast<uint8_t*>(is_v ? p.V : p.K) + at * d;
            for (int c = lane; c < d; c += 32)
                y[c] = __nv_cvt_float_to_fp8(__fmul_rn(__bfloat162float(x[c]), inv), __NV_SATFINITE, __NV_E4M3);
            if (lane == 0) (is_v ? p.v_scale : p.k_scale)[at] = __fdiv_rn(amax, kE4M3Max);
        }
    }
}

// One warp per (sequence, position, KV head, K or V).
template <bool E4M3>
__global__ void __launch_bounds__(256) kv_read_kernel(const KvParams p) {
    pdl_trigger();
    pdl_wait();
    const int lane = threadIdx.x & 31;
    const int k = p.v.kv_heads, d = p.v.d;
    const long long n_items = static_cast<long long>(p.v.n_seqs) * p.max_len * k * 2;
    const long long warps = static_cast<long long>(gridDim.x) * 8;
    for (long long it = static_cast<long long>(blockIdx.x) * 8 + (threadIdx.x >> 5); it < n_items; it += warps) {
        const bool is_v = it & 1;
        const int g = static_cast<int>((it >> 1) % k);
        const long long r = (it >> 1) / k;
        const int s = static_cast<int>(r / p.max_len);
        const long long pos = r % p.max_len;
        if (pos >= p.v.kv_len[s]) continue;
        const long long page = paged_page(p.v, s, static_cast<int>(pos));
        if (page < 0 && lane == 0 && p.status) atomicOr(p.status, kStatusPage);
        const long long at = page < 0 ? 0 : paged_row(p.v, page, g, static_cast<int>(pos));
        __nv_bfloat16* y = (is_v ? p.v_out : p.k_out) + (r * k + g) * d;
        for (int c = lane; c < d; c += 32) {
            float x = 0.0f;
            if (page >= 0) {
                if constexpr (E4M3) {
                    const uint8_t code = static_cast<const uint8_t*>(is_v ? p.V : p.K)[at * d + c];
                    x = __half2float(__half(__nv_cvt_fp8_to_halfraw(code, __NV_E4M3))) *
                        (is_v ? p.v_scale : p.k_scale)[at];
                } else {
                    x = __bfloat162float(static_cast<const __nv_bfloat16*>(is_v ? p.V : p.K)[at * d + c]);
                }
            }
            y[c] = __float2bfloat16_rn(x);
        }
    }
}

KvParams params_of(const tpi::PagedArgs& a) {
    KvParams p{};
    p.v = tpi::paged_view(a);
    p.K = a.K;
    p.V = a.V;
    p.k_scale = a.k_scale;
    p.v_scale = a.v_scale;
    p.qkv = static_cast<const __nv_bfloat16*>(a.QKV);
    p.ld_qkv = a.ld_qkv;
    p.shard_w = static_cast<int>(a.shard_w);
    p.q_w = static_cast<int>(a.q_w);
    p.kv_w = static_cast<int>(a.kv_w);
    p.kv_per_shard = a.kv_heads / a.t;
    p.t = a.t;
    p.status = a.status;
    return p;
}

int launched(const char* what, cudaError_t e, std::string* err) {
    if (e == cudaSuccess) e = cudaGetLastError();
    if (e == cudaSuccess) return TP_OK;
    if (err) *err = std::string(what) + ": " + cudaGetErrorString(e);
    return TP_ERR_CUDA;
}

unsigned blocks_for(long long warps) {
    const long long most = static_cast<long long>(tpi::device_sm_count()) * 8;
    const long long need = (warps + 7) / 8;
    return static_cast<unsigned>(need < most ? need : most);
}

}  // namespace

namespace tpi {

int kv_write_launch(const PagedArgs& a, cudaStream_t stream, std::string* err) {
    if (a.n_seqs == 0) return TP_OK;
    const KvParams p = params_of(a);
    const unsigned grid = blocks_for(a.tokens * a.kv_heads * 2);
    const cudaError_t e = a.e4m3 ? launch_pdl(kv_write_kernel<true>, dim3(grid), dim3(256), 0, stream, p)
                                 : launch_pdl(kv_write_kernel<false>, dim3(grid), dim3(256), 0, stream, p);
    return launched("cache write kernel", e, err);
}

int kv_read_launch(const PagedArgs& a, int64_t max_len, void* k_out, void* v_out, cudaStream_t stream,
                   std::string* err) {
    if (a.n_seqs == 0 || max_len == 0) return TP_OK;
    KvParams p = params_of(a);
    p.max_len = max_len;
    p.k_out = static_cast<__nv_bfloat16*>(k_out);
    p.v_out = static_cast<__nv_bfloat16*>(v_out);
    const unsigned grid = blocks_for(static_cast<long long>(a.n_seqs) * max_len * a.kv_heads * 2);
    const cudaError_t e = a.e4m3 ? launch_pdl(kv_read_kernel<true>, dim3(grid), dim3(256), 0, stream, p)
                                 : launch_pdl(kv_read_kernel<false>, dim3(grid), dim3(256), 0, stream, p);
    return launched("cache read kernel", e, err);
}

}  // namespace tpi
