// tp_layernorm.cu -- layer norm with a gain and a bias, and its gradients.
//
// Source: "텐서 병렬화" (itwiki, Tensor parallelism), section "통신 연산 f와
// g": norms are replicated, so every shard's norm is this one.  With
// mu = mean_j x_j, r = 1 / sqrt(mean_j (x_j - mu)^2 + eps), xh = (x - mu) r:
//   y      = xh gain + bias
//   dx     = dres + r (g - mean_j g_j - xh mean_j g_j xh_j),   g = dy gain
//   dgain  = sum over rows of dy xh,   dbias = sum over rows of dy
//
// Both directions have to move their rows once.  A CTA strides over the rows,
// GROUPS of them at a time, each on W warps with VPT 16-byte pieces a thread; the
// next rows are on their way to shared memory meanwhile (Ring), and the gain and
// the bias lie there as fp32.  A row's statistics take one exchange between its
// warps.  The weights' gradients are summed in registers over a CTA's rows, and a
// second kernel adds the CTAs' sums in a fixed order: no atomics, so repeated calls
// give the same bits.
//
// Measured (the bytes' time at the copy rate in brackets): forward 8192 x 4096
// 23.8 us (19.8), 16384 x 768 10.3 (7.4), 2000 x 12288 23.5 (14.5); gradients 8192 x
// 4096 43.8 (29.7), 2048 x 1024 9 to 11 (1.9), 3001 x 2568 with a residual 22.2 (9.1).
// The forward kernel is at the memory's rate once it runs (16384 x 4096: 6.4 TB/s of
// 268 MB), what is above that is the launch and the first rows.  The gradients' kernel
// issues in half of all cycles with 16 warps on an SM (two sums of a column for every
// value held leave no registers for more), and its weights' part costs 5 us: the
// CTA's sums to memory, a launch, and the sum over 152 CTAs.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <string>
#include <type_traits>

#include "tp_device.cuh"
#include "tp_internal.h"
#include "tp_packed.cuh"

namespace {

using namespace tpk;

constexpr int MAX_PARTS = 512;  // most CTAs of the gradients' kernel

__device__ __forceinline__ uint4 zeros8() { return make_uint4(0u, 0u, 0u, 0u); }

// Eight bf16 values as four pairs of fp32, and back.
__device__ __forceinline__ void unpack8(const uint4& u, uint64_t (&p)[4]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = unpack_bf16x2(w[i]);
        p[i] = f2_pack(f.x, f.y);
    }
}
__device__ __forceinline__ uint4 pack8(const uint64_t (&p)[4]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float lo, hi;
        f2_unpack(p[i], lo, hi);
        w[i] = pack_bf16x2(lo, hi);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ uint64_t both(float x) { return f2_pack(x, x); }
__device__ __forceinline__ float sum2(uint64_t p) {
    float lo, hi;
    f2_unpack(p, lo, hi);
    return lo + hi;
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// The gain (or the bias) as fp32 in shared memory, so that a row costs neither
// its conversion nor the choice of a default: the first four values of piece v at
// [v], the other four at [nv + v], free of bank conflicts.
__device__ __forceinline__ void stage_weights(const __nv_bfloat16* from, float value, int nv, float4* to) {
    for (int v = threadIdx.x; v < nv; v += blockDim.x) {
        float4 a = make_float4(value, value, value, value), b = a;
        if (from) {
            const uint4 u = reinterpret_cast<const uint4*>(from)[v];
            const float2 f0 = unpack_bf16x2(u.x), f1 = unpack_bf16x2(u.y), f2 = unpack_bf16x2(u.z), f3 = unpack_bf16x2(u.w);
            a = make_float4(f0.x, f0.y, f1.x, f1.y);
            b = make_float4(f2.x, f2.y, f3.x, f3.y);
        }
        to[v] = a;
        to[nv + v] = b;
    }
}
__device__ __forceinline__ void weights8(const float4* from, int nv, int v, uint64_t (&p)[4]) {
    const float4 a = from[v], b = from[nv + v];
    p[0] = f2_pack(a.x, a.y);
    p[1] = f2_pack(a.z, a.w);
    p[2] = f2_pack(b.x, b.y);
    p[3] = f2_pack(b.z, b.w);
}

// A row's pieces: W warps, VPT a thread, nv in all; this thread's are first,
// first + 32 W, ...  count(w): the values that warp w holds.  FULL: rows of just
// as many pieces as there are places; with up to four a thread, all but the last
// are there in any case (for_fill sees to it).
template <int W, int VPT, bool FULL>
struct Pieces {
    int first, nv;
    __device__ __forceinline__ explicit Pieces(int h) : first(threadIdx.x % (32 * W)), nv(h >> 3) {}
    __device__ __forceinline__ bool has(int i) const { return FULL || (VPT <= 4 && i + 1 < VPT) || first + i * 32 * W < nv; }
    __device__ __forceinline__ int at(int i) const { return first + i * 32 * W; }
    __device__ __forceinline__ float count(int w) const {
        if (FULL) return 256.0f * VPT;
        int n = 0;
#pragma unroll
        for (int i = 0; i < VPT; ++i) n += min(max(nv - (i * W + w) * 32, 0), 32);
        return static_cast<float>(n * 8);
    }
};

// Rows on their way to shared memory: ARRAYS of them at a time, STAGES deep.  A
// thread copies and reads its own pieces, so no barrier guards them; what lies
// past a row's end stays zero.  A stage is filled again after what was read from
// it has been used.
template <int VPT, int ARRAYS, int STAGES, int THREADS>
struct Ring {
    static constexpr int PIECES = STAGES * ARRAYS * VPT * THREADS;
    uint4* mine;
    __device__ __forceinline__ explicit Ring(uint4* shared) : mine(shared + threadIdx.x) {
#pragma unroll
        for (int i = 0; i < PIECES / THREADS; ++i) mine[i * THREADS] = zeros8();
    }
    __device__ __forceinline__ uint4& at(int stage, int array, int i) const {
        return mine[((stage * ARRAYS + array) * VPT + i) * THREADS];
    }
    template <typename P>
    __device__ __forceinline__ void copy(const P& p, int stage, int array, const __nv_bfloat16* row) const {
#pragma unroll
        for (int i = 0; i < VPT; ++i)
            if (p.has(i))
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(&at(stage, array, i))),
                             "l"(reinterpret_cast<const uint4*>(row) + p.at(i))
                             : "memory");
    }
    static __device__ __forceinline__ void commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
    static __device__ __forceinline__ void wait() {  // all of this thread's copies but those of the last STAGES - 1 commits
        asm volatile("cp.async.wait_group %0;" ::"n"(STAGES - 1) : "memory");
    }
};

// N values of each of a row's W warps, brought together in shared memory: two
// slots in turn, so that one barrier a row is enough.  Lane k gets those of warp
// k % W; all(x) adds x over the warps.
template <int W, int N>
struct Exchange {
    float* at;
    int turn = 0;
    __device__ __forceinline__ explicit Exchange(float* shared) : at(shared + threadIdx.x / (32 * W) * 2 * W * N) {}
    __device__ __forceinline__ void operator()(float (&v)[N]) {
        if (W == 1) return;
        float* slot = at + turn * W * N;
        if ((threadIdx.x & 31) == 0) {
#pragma unroll
            for (int i = 0; i < N; ++i) slot[threadIdx.x / 32 % W * N + i] = v[i];
        }
        named_bar_sync(1 + threadIdx.x / (32 * W), 32 * W);
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = slot[threadIdx.x % W * N + i];
        turn ^= 1;
    }
    static __device__ __forceinline__ float all(float x) {
#pragma unroll
        for (int o = W / 2; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
        return x;
    }
};

// The mean of a warp's values and the sum of their squared distances from it:
// no difference of large sums, so a row whose mean is far from zero keeps its
// variance.
template <int VPT, typename P, typename F>
__device__ __forceinline__ float2 warp_moments(const P& p, float inv_count, F&& piece) {
    uint64_t s = both(0.0f), x[4];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        piece(i, x);  // pieces past the row hold zeros
        s = f2_add(s, f2_add(f2_add(x[0], x[1]), f2_add(x[2], x[3])));
    }
    const float mean = warp_sum(sum2(s)) * inv_count;
    uint64_t a = both(0.0f), b = both(0.0f);
    const uint64_t off = both(-mean);
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        if (!p.has(i)) continue;
        piece(i, x);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            x[e] = f2_add(x[e], off);
            if (e & 1) a = f2_fma(x[e], x[e], a);
            else b = f2_fma(x[e], x[e], b);
        }
    }
    return make_float2(mean, warp_sum(sum2(a) + sum2(b)));
}

// A row's mean and 1 / sqrt(variance + eps) from its warps' moments (lane k has
// those of warp k % W, and that warp's share of the row).
template <int W, int N>
__device__ __forceinline__ float2 row_stats(float warp_mean, float m2, float share, float inv_h, float eps) {
    using X = Exchange<W, N>;
    const float mean = W == 1 ? warp_mean : X::all(share * warp_mean), d = warp_mean - mean;
    return make_float2(mean, rsqrtf(X::all(fmaf(share * d, d, m2 * inv_h)) + eps));
}

template <int W, int VPT>
struct Forward {
    static constexpr int THREADS = 256, CTAS = VPT > 4 ? 1 : W > 4 ? 2 : 3, STAGES = 2;  // CTAs an SM
    static constexpr int GROUPS = THREADS / (32 * W);                                    // rows of a CTA at a time
    using Rows = Ring<VPT, 1, STAGES, THREADS>;
    static size_t shared_bytes(int h) { return (Rows::PIECES + h / 2) * sizeof(uint4); }
};

template <int W, int VPT, bool FULL>
__global__ void __launch_bounds__(Forward<W, VPT>::THREADS, Forward<W, VPT>::CTAS)
    layernorm_kernel(const __nv_bfloat16* x, long long rows, int h, const __nv_bfloat16* gain,
                     const __nv_bfloat16* bias, float eps, __nv_bfloat16* y, float* stats) {
    using C = Forward<W, VPT>;
    __shared__ float shared[C::GROUPS * 2 * W * 2];
    extern __shared__ uint4 dynamic[];
    pdl_trigger();
    pdl_wait();
    const Pieces<W, VPT, FULL> p(h);
    const typename C::Rows ring(dynamic);
    Exchange<W, 2> exchange(shared);
    const float inv_h = 1.0f / static_cast<float>(h), share = p.count(threadIdx.x % W) * inv_h;
    const float inv_count = 1.0f / fmaxf(p.count(threadIdx.x / 32 % W), 1.0f);
    const long long step = static_cast<long long>(gridDim.x) * C::GROUPS;
    long long row = static_cast<long long>(blockIdx.x) * C::GROUPS + threadIdx.x / (32 * W);
    auto load = [&](long long r, int stage) {
        if (r < rows) ring.copy(p, stage, 0, x + r * h);
        ring.commit();
    };
#pragma unroll
    for (int k = 0; k < C::STAGES; ++k) load(row + k * step, k);
    float4* weights = reinterpret_cast<float4*>(dynamic + C::Rows::PIECES);  // gain, bias
    stage_weights(gain, 1.0f, p.nv, weights);
    stage_weights(bias, 0.0f, p.nv, weights + 2 * p.nv);
    __syncthreads();
    for (int stage = 0; row < rows; row += step, stage ^= 1) {
        ring.wait();
        uint64_t f[VPT][4];
#pragma unroll
        for (int i = 0; i < VPT; ++i) unpack8(ring.at(stage, 0, i), f[i]);
        const float2 m = warp_moments<VPT>(p, inv_count, [&](int i, uint64_t(&out)[4]) {
#pragma unroll
            for (int e = 0; e < 4; ++e) out[e] = f[i][e];
        });
        load(row + C::STAGES * step, stage);
        float v[2] = {m.x, m.y};
        exchange(v);
        const float2 st = row_stats<W, 2>(v[0], v[1], share, inv_h, eps);
        if (stats && p.first == 0) {
            stats[row] = st.x;
            stats[rows + row] = st.y;
        }
        const uint64_t off = both(-st.x), r = both(st.y);
        uint4* out = reinterpret_cast<uint4*>(y + row * h);
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            if (!p.has(i)) continue;
            uint64_t g[4], b[4];
            weights8(weights, p.nv, p.at(i), g);
            weights8(weights + 2 * p.nv, p.nv, p.at(i), b);
#pragma unroll
            for (int e = 0; e < 4; ++e) f[i][e] = f2_fma(f2_mul(f2_add(f[i][e], off), r), g[e], b[e]);
            out[p.at(i)] = pack8(f[i]);
        }
    }
}

template <int W, int VPT>
struct Backward {
    // One CTA an SM: its rows' sums leave as one part.  Rows above 8192 leave room
    // for one stage alone.
    static constexpr int THREADS = 512, STAGES = W > 8 && VPT > 2 ? 1 : 2;
    static constexpr bool HOLD = VPT <= 2;
    static constexpr int GROUPS = THREADS / (32 * W);
    using Rows = Ring<VPT, 3, STAGES, THREADS>;  // x, dy, dres
    static size_t shared_bytes(int h) { return (Rows::PIECES + h / 4) * sizeof(uint4); }
    // The sums of columns at the end take the ring's place.
    static_assert(Rows::PIECES * 16 >= GROUPS * 32 * W * VPT * 8 * 4, "");
};

// dx of every row, and the CTA's sums for dgain and dbias in parts
// [CTAs][2][h].  dx may be dy or dres: no row's inputs are read after its outputs
// are stored, and no two threads read or store the same piece.  The sums over a
// row are taken about the warps' own means, so that they need one exchange with
// those that give the statistics:
//   sum g xh = r sum_w (sum g (x - mean_w) + (mean_w - mu) sum g).
template <int W, int VPT, bool FULL>
__global__ void __launch_bounds__(Backward<W, VPT>::THREADS, 1)
    layernorm_bwd_kernel(const __nv_bfloat16* x, long long rows, int h, const __nv_bfloat16* gain, float eps,
                         const float* stats, const __nv_bfloat16* dy, const __nv_bfloat16* dres,
                         __nv_bfloat16* dx, float* parts) {
    using C = Backward<W, VPT>;
    constexpr bool HOLD = C::HOLD;
    __shared__ float shared[C::GROUPS * 2 * W * 4];
    extern __shared__ uint4 dynamic[];
    pdl_trigger();
    pdl_wait();
    const Pieces<W, VPT, FULL> p(h);
    const typename C::Rows ring(dynamic);
    Exchange<W, 4> exchange(shared);
    const int group = threadIdx.x / (32 * W);
    const float inv_h = 1.0f / static_cast<float>(h), share = p.count(threadIdx.x % W) * inv_h;
    const float inv_count = 1.0f / fmaxf(p.count(threadIdx.x / 32 % W), 1.0f);
    const long long step = static_cast<long long>(gridDim.x) * C::GROUPS;
    long long row = static_cast<long long>(blockIdx.x) * C::GROUPS + group;
    auto load = [&](long long r, int stage) {
        if (r < rows) {
            ring.copy(p, stage, 0, x + r * h);
            ring.copy(p, stage, 1, dy + r * h);
            if (dres) ring.copy(p, stage, 2, dres + r * h);
        }
        ring.commit();
    };
    auto saved_at = [&](long long r) {
        return stats && r < rows ? make_float2(stats[r], stats[rows + r]) : make_float2(0.0f, 0.0f);
    };
#pragma unroll
    for (int k = 0; k < C::STAGES; ++k) load(row + k * step, k);
    float2 snext = saved_at(row);
    float4* weights = reinterpret_cast<float4*>(dynamic + C::Rows::PIECES);  // gain
    stage_weights(gain, 1.0f, p.nv, weights);
    uint64_t dg[VPT][4], db[VPT][4];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
#pragma unroll
        for (int e = 0; e < 4; ++e) dg[i][e] = db[i][e] = both(0.0f);
    }
    __syncthreads();
    for (int stage = 0; row < rows; row += step, stage = (stage + 1) % C::STAGES) {
        const float2 saved = snext;
        snext = saved_at(row + step);
        ring.wait();
        // Up to two pieces a thread stay unpacked in registers; more are read and
        // unpacked again (twelve values each of x, dy and the two sums would spill).
        uint64_t xk[HOLD ? VPT : 1][4], dk[HOLD ? VPT : 1][4];
        if (HOLD) {
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                unpack8(ring.at(stage, 0, i), xk[HOLD ? i : 0]);
                unpack8(ring.at(stage, 1, i), dk[HOLD ? i : 0]);
            }
        }
        auto piece = [&](int i, int array, uint64_t(&out)[4]) {
            if (HOLD) {
#pragma unroll
                for (int e = 0; e < 4; ++e) out[e] = array ? dk[HOLD ? i : 0][e] : xk[HOLD ? i : 0][e];
            } else {
                unpack8(ring.at(stage, array, i), out);
            }
        };
        const float2 m = stats ? make_float2(saved.x, 0.0f)
                               : warp_moments<VPT>(p, inv_count, [&](int i, uint64_t(&out)[4]) { piece(i, 0, out); });
        uint64_t sg = both(0.0f), sgx = both(0.0f);
        uint64_t off = both(-m.x);
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            if (!p.has(i)) continue;
            uint64_t f[4], g[4], d[4];
            piece(i, 0, f);
            piece(i, 1, d);
            weights8(weights, p.nv, p.at(i), g);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                g[e] = f2_mul(g[e], d[e]);
                sg = f2_add(sg, g[e]);
                sgx = f2_fma(g[e], f2_add(f[e], off), sgx);
            }
        }
        float v[4] = {m.x, m.y, warp_sum(sum2(sg)), warp_sum(sum2(sgx))};
        exchange(v);
        using X = Exchange<W, 4>;
        const float2 st = stats ? saved : row_stats<W, 4>(v[0], v[1], share, inv_h, eps);
        const float c1 = X::all(v[2]) * inv_h, c2 = X::all(fmaf(v[0] - st.x, v[2], v[3])) * (inv_h * st.y);
        const uint64_t r = both(st.y), n1 = both(-c1), n2 = both(-c2);
        off = both(-st.x);
        uint4* out = reinterpret_cast<uint4*>(dx + row * h);
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            if (!p.has(i)) continue;
            uint64_t f[4], g[4], d[4], a[4];
            piece(i, 0, f);
            piece(i, 1, d);
            weights8(weights, p.nv, p.at(i), g);
            unpack8(ring.at(stage, 2, i), a);  // zeros without dres
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                f[e] = f2_mul(f2_add(f[e], off), r);
                dg[i][e] = f2_fma(d[e], f[e], dg[i][e]);
                db[i][e] = f2_add(db[i][e], d[e]);
                a[e] = f2_fma(r, f2_fma(f[e], n2, f2_fma(d[e], g[e], n1)), a[e]);
            }
            out[p.at(i)] = pack8(a);
        }
        load(row + C::STAGES * step, stage);
    }
    if (!parts) return;
    // The rows that the CTA holds at a time are added in shared memory.
    __syncthreads();
    float2* cols = reinterpret_cast<float2*>(dynamic);  // [GROUPS][h / 2] pairs of columns
    float2* out = reinterpret_cast<float2*>(parts + static_cast<long long>(blockIdx.x) * 2 * h);
    const int half = h >> 1;
#pragma unroll
    for (int k = 0; k < 2; ++k) {  // dgain, dbias
        float2* mine = C::GROUPS > 1 ? cols + group * half : out + k * half;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            if (!p.has(i)) continue;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                float2 s;
                f2_unpack(k ? db[i][e] : dg[i][e], s.x, s.y);
                mine[p.at(i) * 4 + e] = s;
            }
        }
        if (C::GROUPS == 1) continue;
        __syncthreads();
        for (int c = threadIdx.x; c < half; c += C::THREADS) {
            float2 s = cols[c];
#pragma unroll
            for (int g = 1; g < C::GROUPS; ++g) {
                s.x += cols[g * half + c].x;
                s.y += cols[g * half + c].y;
            }
            out[k * half + c] = s;
        }
        __syncthreads();
    }
}

// dgain (+)= and dbias (+)= the CTAs' sums in a fixed order: 32 columns a CTA,
// warps that take every JOIN_WARPS-th part, joined in order.
constexpr int JOIN_WARPS = 16;

__global__ void __launch_bounds__(JOIN_WARPS * 32) layernorm_join_kernel(const float* parts, int n, int h,
                                                                        float* dgain, float* dbias, int accumulate) {
    pdl_trigger();
    pdl_wait();
    __shared__ float sum[JOIN_WARPS][32];
    float* out = blockIdx.y ? dbias : dgain;
    if (!out) return;
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
    float s = 0.0f;
    // All of a warp's loads at once: with eight and the rest one by one the rest
    // waited for memory as long as the eight, each.
    constexpr int LOADS = 10;
    for (int k0 = w; c < h && k0 < n; k0 += JOIN_WARPS * LOADS) {
        float v[LOADS];
#pragma unroll
        for (int i = 0; i < LOADS; ++i) {
            const int k = k0 + i * JOIN_WARPS;
            v[i] = k < n ? parts[(static_cast<long long>(k) * 2 + blockIdx.y) * h + c] : 0.0f;
        }
#pragma unroll
        for (int i = 0; i < LOADS; ++i) s += v[i];
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

// Raises a kernel's limit on dynamic shared memory to what any row takes, once a
// device.
constexpr int MOST_SHARED = 227 * 1024 - 2048;
template <auto KERNEL>
int allow_shared(std::string* err) {
    static bool done[64] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) == cudaSuccess && dev >= 0 && dev < 64 && done[dev]) return TP_OK;
    if (cudaFuncSetAttribute(KERNEL, cudaFuncAttributeMaxDynamicSharedMemorySize, MOST_SHARED) != cudaSuccess)
        return check("layer norm's shared memory", err);
    if (dev >= 0 && dev < 64) done[dev] = true;
    return TP_OK;
}

template <int N>
using Int = std::integral_constant<int, N>;
// Rows of LEAST to NV pieces.
template <int W, int VPT, int LEAST, int NV, typename F>
int for_fill(int nv, F&& f) {
    static_assert(NV == 32 * W * VPT && (VPT > 4 || LEAST >= 32 * W * (VPT - 1)), "");
    return nv == NV ? f(Int<W>(), Int<VPT>(), std::true_type()) : f(Int<W>(), Int<VPT>(), std::false_type());
}

// Warps of a row and 16-byte pieces a thread for rows of h.  Forward: as many
// pieces a thread as keep three CTAs on an SM, since what a warp does once a row
// costs as much as 20 values (16384 x 768: 10.3 us with three pieces, 11.2 with four
// places).
template <typename F>
int for_forward(int h, F&& f) {
    const int nv = h / 8;
    if (nv <= 32) return for_fill<1, 1, 0, 32>(nv, f);
    if (nv <= 64) return for_fill<1, 2, 33, 64>(nv, f);
    if (nv <= 96) return for_fill<1, 3, 65, 96>(nv, f);
    if (nv <= 128) return for_fill<1, 4, 97, 128>(nv, f);
    if (nv <= 192) return for_fill<2, 3, 129, 192>(nv, f);
    if (nv <= 256) return for_fill<2, 4, 193, 256>(nv, f);
    if (nv <= 384) return for_fill<4, 3, 257, 384>(nv, f);
    if (nv <= 512) return for_fill<4, 4, 385, 512>(nv, f);
    if (nv <= 768) return for_fill<8, 3, 513, 768>(nv, f);
    if (nv <= 1024) return for_fill<8, 4, 769, 1024>(nv, f);
    if (nv <= 1536) return for_fill<8, 6, 1025, 1536>(nv, f);
    return for_fill<8, 8, 1537, 2048>(nv, f);
}
// Backward: two pieces a thread, three where they fill the places better (3001 x
// 2568: 23.0 us on four warps of three pieces, 24.2 on eight of two; 4096 x 5000:
// 34 and 39 us; but 8192 x 768: 22 us on one warp, 17 on two).
template <typename F>
int for_backward(int h, F&& f) {
    const int nv = h / 8;
    if (nv <= 32) return for_fill<1, 1, 0, 32>(nv, f);
    if (nv <= 64) return for_fill<1, 2, 33, 64>(nv, f);
    if (nv <= 128) return for_fill<2, 2, 65, 128>(nv, f);
    if (nv <= 256) return for_fill<4, 2, 129, 256>(nv, f);
    if (nv <= 384) return for_fill<4, 3, 257, 384>(nv, f);
    if (nv <= 512) return for_fill<8, 2, 385, 512>(nv, f);
    if (nv <= 768) return for_fill<8, 3, 513, 768>(nv, f);
    if (nv <= 1024) return for_fill<16, 2, 769, 1024>(nv, f);
    if (nv <= 1536) return for_fill<16, 3, 1025, 1536>(nv, f);
    return for_fill<16, 4, 1537, 2048>(nv, f);
}

}  // namespace

namespace tpi {

int layernorm_launch(const void* x, int64_t rows, int h, const void* gain, const void* bias, float eps, void* y,
                     float* stats, cudaStream_t stream, std::string* err) {
    if (rows == 0) return TP_OK;
    return for_forward(h, [&](auto W, auto VPT, auto FULL) {
        using C = Forward<decltype(W)::value, decltype(VPT)::value>;
        constexpr auto kern = layernorm_kernel<decltype(W)::value, decltype(VPT)::value, decltype(FULL)::value>;
        const int rc = allow_shared<kern>(err);
        if (rc) return rc;
        const int64_t grid = std::min<int64_t>((rows + C::GROUPS - 1) / C::GROUPS, device_sm_count() * C::CTAS);
        launch_pdl(kern, dim3((unsigned)grid), dim3(C::THREADS), C::shared_bytes(h), stream,
                   static_cast<const __nv_bfloat16*>(x), static_cast<long long>(rows), h,
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
        const int rc = for_backward(h, [&](auto W, auto VPT, auto FULL) {
            using C = Backward<decltype(W)::value, decltype(VPT)::value>;
            constexpr auto kern = layernorm_bwd_kernel<decltype(W)::value, decltype(VPT)::value, decltype(FULL)::value>;
            const int rc = allow_shared<kern>(err);
            if (rc) return rc;
            grid = std::min<int64_t>({(rows + C::GROUPS - 1) / C::GROUPS, device_sm_count(), MAX_PARTS});
            launch_pdl(kern, dim3((unsigned)grid), dim3(C::THREADS), C::shared_bytes(h), stream,
                       static_cast<const __nv_bfloat16*>(x), static_cast<long long>(rows), h,
                       static_cast<const __nv_bfloat16*>(gain), eps, stats, static_cast<const __nv_bfloat16*>(dy),
                       static_cast<const __nv_bfloat16*>(dres), static_cast<__nv_bfloat16*>(dx),
                       weights ? static_cast<float*>(scratch) : nullptr);
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
