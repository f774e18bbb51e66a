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
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <string>

#include "tp_device.cuh"
#include "tp_internal.h"

namespace {

using namespace tpk;

constexpr int VT = 512;
constexpr float LOG2E = 1.4426950408889634f;

struct VerifyParams {
    const __nv_bfloat16 *z, *y;
    long long rows, v;
    const int32_t *ids, *q_start;
    const float *temperature, *u, *noise;
    int32_t *accepted, *tokens;
    int n_seqs;
};

// Largest value and its lowest index.
struct Best {
    float v;
    int i;
};
__device__ __forceinline__ Best better(Best a, Best b) {
    return (b.v > a.v || (b.v == a.v && b.i < a.i)) ? b : a;
}

__device__ __forceinline__ Best block_best(Best a, Best* red) {
    for (int o = 16; o > 0; o >>= 1) {
        Best b = {__shfl_xor_sync(0xffffffffu, a.v, o), __shfl_xor_sync(0xffffffffu, a.i, o)};
        a = better(a, b);
    }
    __syncthreads();
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = a;
    __syncthreads();
    a = red[0];
    for (int w = 1; w < VT / 32; ++w) a = better(a, red[w]);
    return a;
}

// m = max_v x_v and sum_v 2^((x_v - m) it), it = log2(e) / T: the difference
// comes first, so that logits at the type's ends do not overflow.
__device__ __forceinline__ float2 row_stats(const __nv_bfloat16* x, long long v, float it, float* red) {
    float m = -INFINITY;
    for (long long c = threadIdx.x; c < v; c += VT) m = fmaxf(m, __bfloat162float(x[c]));
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    __syncthreads();
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = m;
    __syncthreads();
    for (int w = 0; w < VT / 32; ++w) m = fmaxf(m, red[w]);
    float s = 0.0f;
    if (m > -INFINITY)
        for (long long c = threadIdx.x; c < v; c += VT) s += exp2f((__bfloat162float(x[c]) - m) * it);
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = s;
    __syncthreads();
    s = 0.0f;
    for (int w = 0; w < VT / 32; ++w) s += red[w];
    return make_float2(m, s);
}

__device__ __forceinline__ float prob(float x, float it, float2 st) {
    return st.y > 0.0f ? exp2f((x - st.x) * it) / st.y : 0.0f;
}

// One CTA per sequence.
__global__ void __launch_bounds__(VT) verify_simple_kernel(const VerifyParams p) {
    pdl_trigger();
    pdl_wait();
    __shared__ float red[VT / 32];
    __shared__ Best bred[VT / 32];
    const int s = blockIdx.x;
    const long long r0 = min(max(static_cast<long long>(p.q_start[s]), 0ll), p.rows);
    const long long r1 = min(max(static_cast<long long>(p.q_start[s + 1]), r0), p.rows);
    const int n = static_cast<int>(r1 - r0);
    const float T = p.temperature ? p.temperature[s] : 1.0f;
    const bool greedy = !(T > 0.0f);
    const float it = fminf(LOG2E / T, 1e30f);  // finite, so that 0 * it is 0
    int taken = 0, token = -1;
    for (int i = 0; i < n; ++i) {
        const __nv_bfloat16* z = p.z + (r0 + i) * p.v;
        const __nv_bfloat16* y = (p.y && i + 1 < n) ? p.y + (r0 + i) * p.v : nullptr;
        const long long x = i + 1 < n ? p.ids[r0 + i + 1] : -1;
        const bool inside = x >= 0 && x < p.v;
        Best b = {-INFINITY, 0x7fffffff};
        if (greedy) {
            for (long long c = threadIdx.x; c < p.v; c += VT)
                b = better(b, Best{__bfloat162float(z[c]), static_cast<int>(c)});
            b = block_best(b, bred);
            token = b.v > -INFINITY ? b.i : -1;
            if (i + 1 < n && inside && token == x) {
                ++taken;
                continue;
            }
            break;
        }
        const float2 sp = row_stats(z, p.v, it, red);
        float2 sq = make_float2(0.0f, 0.0f);
        if (y) sq = row_stats(y, p.v, it, red);
        if (inside) {
            const float px = prob(__bfloat162float(z[x]), it, sp);
            const float qx = y ? prob(__bfloat162float(y[x]), it, sq) : 0.0f;
            if (p.u[r0 + i] * qx < px) {
                ++taken;
                continue;
            }
        }
        Best f = b;  // from p alone, where max(0, p - q) leaves nothing
        for (long long c = threadIdx.x; c < p.v; c += VT) {
            const float e = p.noise ? p.noise[s * p.v + c] : 1.0f;
            const float pc = prob(__bfloat162float(z[c]), it, sp);
            const float w = y ? pc - prob(__bfloat162float(y[c]), it, sq) : pc;
            if (w > 0.0f) b = better(b, Best{w / e, static_cast<int>(c)});
            if (pc > 0.0f) f = better(f, Best{pc / e, static_cast<int>(c)});
        }
        b = block_best(b, bred);
        f = block_best(f, bred);
        if (!(b.v > 0.0f)) b = f;
        token = b.v > 0.0f ? b.i : -1;
        break;
    }
    if (threadIdx.x == 0) p.accepted[s] = taken;
    for (int i = threadIdx.x; i < n; i += VT)
        p.tokens[r0 + i] = i < taken ? p.ids[r0 + i + 1] : i == taken ? token : -1;
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
    p.n_seqs = a.n_seqs;
    cudaError_t e = launch_pdl(verify_simple_kernel, dim3(static_cast<unsigned>(a.n_seqs)), dim3(VT), 0, stream, p);
    if (e == cudaSuccess) e = cudaGetLastError();
    if (e != cudaSuccess) {
        if (err) *err = std::string("verification kernel: ") + cudaGetErrorString(e);
        return TP_ERR_CUDA;
    }
    return TP_OK;
}

}  // namespace tpi
