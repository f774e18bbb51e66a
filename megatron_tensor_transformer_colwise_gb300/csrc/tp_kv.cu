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
//
// Both directions are bound by memory: every element is read and written once.
// A row of d bf16 (128 or 256 bytes) is a group of d / 16 lanes, two pieces of 16
// bytes each (pieces c and c + d / 16, so that each access of a group is contiguous):
// a warp moves 4 or 8 rows at a time.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <string>

#include "tp_device.cuh"
#include "tp_internal.h"
#include "tp_paged.cuh"

namespace {

using namespace tpk;

constexpr float kE4M3Max = 448.0f;
constexpr float kAmaxFloor = 7.888609052210118e-31f;  // 2^-100
constexpr float kAmaxCeil = 3.3895313892515355e38f;   // largest finite bf16
constexpr int THREADS = 256;
constexpr int STARTS = 1025;  // sequences' starts staged in shared memory, at most

struct KvParams {
    PagedView v;
    void *K, *V;
    float *k_scale, *v_scale;
    const __nv_bfloat16* qkv;
    long long ld_qkv;
    int shard_w, q_w, kv_w, held, heads_step;  // held: KV heads of a shard; heads_step: shards that share one (k < t), else 0
    int log2_k;  // of the KV heads, -1 if that is no power of two
    unsigned* status;
    // read back
    __nv_bfloat16 *k_out, *v_out;
    long long max_len;
    int chunks;  // blocks of tokens of a sequence
};

// Two fp32 as e4m3 (round to nearest even, at most 448, NaN stays NaN); lo in
// the low byte.
__device__ __forceinline__ uint32_t pack_e4m3x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ float2 unpack_e4m3x2(uint32_t codes) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(codes)));
    return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// Two 16-byte pieces of a bf16 row, pieces c and c + LANES of it, to the cache.  at: the cache's row.  The LANES
// lanes of a row call together (amax is theirs).
template <int D, bool E4M3>
__device__ __forceinline__ void store_row(const KvParams& p, bool is_v, long long at, int c, const uint4 (&u)[2], bool live) {
    constexpr int LANES = D / 16;
    if constexpr (!E4M3) {
        uint4* y = reinterpret_cast<uint4*>(is_v ? p.V : p.K) + at * (D / 8) + c;
        if (live) {
            y[0] = u[0];
            y[LANES] = u[1];
        }
    } else {
        const uint32_t w[8] = {u[0].x, u[0].y, u[0].z, u[0].w, u[1].x, u[1].y, u[1].z, u[1].w};
        float x[16], amax = 0.0f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float2 f = unpack_bf16x2(w[e]);
            x[2 * e] = f.x;
            x[2 * e + 1] = f.y;
            amax = fmaxf(amax, fmaxf(fabsf(f.x), fabsf(f.y)));  // NaN is ignored
        }
#pragma unroll
        for (int o = LANES / 2; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
        amax = fminf(fmaxf(amax, kAmaxFloor), kAmaxCeil);
        const float inv = __fdiv_rn(kE4M3Max, amax);
        uint32_t r[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
            r[e] = pack_e4m3x2(__fmul_rn(x[4 * e], inv), __fmul_rn(x[4 * e + 1], inv)) |
                   pack_e4m3x2(__fmul_rn(x[4 * e + 2], inv), __fmul_rn(x[4 * e + 3], inv)) << 16;
        if (live) {
            uint2* y = reinterpret_cast<uint2*>(is_v ? p.V : p.K) + at * (D / 8) + c;
            y[0] = make_uint2(r[0], r[1]);
            y[LANES] = make_uint2(r[2], r[3]);
            if (c == 0) (is_v ? p.v_scale : p.k_scale)[at] = __fdiv_rn(amax, kE4M3Max);
        }
    }
}

// Append.  A group of D / 16 lanes takes a (token, KV head) at a time, K and V
// together: their loads are in flight while the token's place is looked up.  8
// blocks an SM walk the items.  8192 tokens of 8 heads of 128 into 8 bits take
// 8.2 us, the launch included (50 MB at 6.1 TB/s; 11.3 with inputs not in L2).  A
// lane's 32 bytes make that: with 16, and a division by k, the look-ups and quotients
// of twice the lanes kept the schedulers at 0.73 and took 13.1 us.  A block for every
// few tokens with one look-up for all heads took 14.7 to 19.9, since each then
// begins with the whole chain of look-ups.  64 single tokens take 2.5 us, a launch.
template <int D, bool E4M3>
__global__ void __launch_bounds__(THREADS) kv_write_kernel(const __grid_constant__ KvParams p) {
    constexpr int LANES = D / 16;
    pdl_trigger();
    pdl_wait();
    // Every token's owner is looked up: in shared memory, when the sequences' starts fit.
    __shared__ int32_t starts[STARTS];
    const bool staged = p.v.n_seqs < STARTS;
    if (staged) {
        for (int i = threadIdx.x; i <= p.v.n_seqs; i += THREADS) starts[i] = p.v.q_start[i];
        __syncthreads();
    }
    const int c = threadIdx.x % LANES, k = p.v.kv_heads;
    // Below 2^31: the keys and values of as many would be 550 GB.
    const unsigned items = static_cast<unsigned>(p.v.rows) * static_cast<unsigned>(k);
    const unsigned step = gridDim.x * (THREADS / LANES);
    // Whole warps stay in the loop (a row's lanes exchange their maxima).
    for (unsigned base = blockIdx.x * (THREADS / LANES); base < items; base += step) {
        const unsigned it = base + threadIdx.x / LANES;
        const bool in = it < items;
        const int row = static_cast<int>(p.log2_k >= 0 ? (in ? it : 0) >> p.log2_k : (in ? it : 0) / static_cast<unsigned>(k));
        const int g = static_cast<int>((in ? it : 0) - static_cast<unsigned>(row) * k);
        // k >= t: shard g / held holds g; k < t: the first of the shards that share it.
        const int shard = p.heads_step ? g * p.heads_step : p.held == 1 ? g : g / p.held;
        const int local = p.heads_step ? 0 : g - shard * p.held;
        const uint4* x = reinterpret_cast<const uint4*>(p.qkv + row * p.ld_qkv + static_cast<long long>(shard) * p.shard_w +
                                                        p.q_w + local * D) + c;
        const uint4 kx[2] = {x[0], x[LANES]}, vx[2] = {x[p.kv_w / 8], x[p.kv_w / 8 + LANES]};
        const int s = in ? paged_owner(staged ? starts : p.v.q_start, p.v.n_seqs, row) : -1;
        long long at = -1;
        if (s >= 0) {
            const PagedSeq q = paged_seq(p.v, s);
            const int pos = q.len - q.n + (row - q.row0);
            const long long page = paged_page(p.v, s, pos);
            if (page >= 0) at = paged_row(p.v, page, g, pos);
            else if (pos >= 0 && c == 0 && p.status) atomicOr(p.status, kStatusPage);
        }
        store_row<D, E4M3>(p, false, at, c, kx, at >= 0);
        store_row<D, E4M3>(p, true, at, c, vx, at >= 0);
    }
}

// Read back.  Block (chunk, sequence): 16 positions of a sequence, all heads.
// A thread's turn is 32 bytes of bf16 of K and of V of one (position, head), UNROLL
// turns in flight.  16 sequences of 2000 to 16000 positions from 8 bits: 90 us, 6.6
// TB/s; with 64 positions a block 94, with 16 bytes a turn 98.  8 sequences of up to
// 1000 from bf16: 2.5 us, a launch and its chain of loads (3.1 with 64 positions).
constexpr int READ_POS = 16;  // the smallest page: a block's positions share one
template <int D, bool E4M3>
__global__ void __launch_bounds__(THREADS) kv_read_kernel(const __grid_constant__ KvParams p) {
    constexpr int LANES = D / 16, UNROLL = E4M3 ? 4 : 2;
    pdl_trigger();
    pdl_wait();
    const int s = blockIdx.x / p.chunks;
    const long long first = static_cast<long long>(blockIdx.x - s * p.chunks) * READ_POS;
    const long long len = pmin(p.v.kv_len[s], p.max_len);
    const int n = static_cast<int>(pmin(READ_POS, len - first));
    if (n <= 0) return;
    const int c = threadIdx.x % LANES, k = p.v.kv_heads;
    const int items = n * k;
    const long long page = paged_page(p.v, s, static_cast<int>(first));
    if (page < 0 && threadIdx.x == 0 && p.status) atomicOr(p.status, kStatusPage);
    // Items in the cache's order (position fastest within a page and head), so that neighbouring groups read
    // neighbouring rows.
    for (int i0 = threadIdx.x / LANES; i0 < items; i0 += UNROLL * (THREADS / LANES)) {
        uint4 ku[UNROLL][2], vu[UNROLL][2];
        float ks[UNROLL], vs[UNROLL];
        long long to[UNROLL];
#pragma unroll
        for (int e = 0; e < UNROLL; ++e) {
            const int i = i0 + e * (THREADS / LANES);
            to[e] = -1;
            if (i >= items) continue;
            const int g = i / n, pos = i - g * n;
            to[e] = ((s * p.max_len + first + pos) * k + g) * (D / 8) + c;
            ks[e] = vs[e] = 0.0f;
#pragma unroll
            for (int h = 0; h < 2; ++h) ku[e][h] = vu[e][h] = make_uint4(0, 0, 0, 0);
            if (page < 0) continue;
            const long long at = paged_row(p.v, page, g, static_cast<int>(first) + pos);
            if constexpr (E4M3) {
                ks[e] = p.k_scale[at];
                vs[e] = p.v_scale[at];
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const long long x = at * (D / 8) + c + h * LANES;
                if constexpr (E4M3) {
                    const uint2 a = __ldcs(static_cast<const uint2*>(p.K) + x), b = __ldcs(static_cast<const uint2*>(p.V) + x);
                    ku[e][h].x = a.x;
                    ku[e][h].y = a.y;
                    vu[e][h].x = b.x;
                    vu[e][h].y = b.y;
                } else {
                    ku[e][h] = __ldcs(static_cast<const uint4*>(p.K) + x);
                    vu[e][h] = __ldcs(static_cast<const uint4*>(p.V) + x);
                }
            }
        }
#pragma unroll
        for (int e = 0; e < UNROLL; ++e) {
            if (to[e] < 0) continue;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                if constexpr (E4M3) {
                    auto expand = [](uint4 u, float f) {
                        uint32_t r[4];
#pragma unroll
                        for (int x = 0; x < 4; ++x) {
                            const float2 v = unpack_e4m3x2((x < 2 ? u.x : u.y) >> (16 * (x & 1)));
                            r[x] = pack_bf16x2(v.x * f, v.y * f);
                        }
                        return make_uint4(r[0], r[1], r[2], r[3]);
                    };
                    ku[e][h] = expand(ku[e][h], ks[e]);
                    vu[e][h] = expand(vu[e][h], vs[e]);
                }
                __stcs(reinterpret_cast<uint4*>(p.k_out) + to[e] + h * LANES, ku[e][h]);
                __stcs(reinterpret_cast<uint4*>(p.v_out) + to[e] + h * LANES, vu[e][h]);
            }
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
    p.held = a.kv_heads >= a.t ? a.kv_heads / a.t : 1;
    p.heads_step = a.kv_heads >= a.t ? 0 : a.t / a.kv_heads;
    p.log2_k = exact_log2(a.kv_heads);
    p.status = a.status;
    return p;
}

int launched(const char* what, cudaError_t e, std::string* err) {
    if (e == cudaSuccess) e = cudaGetLastError();
    if (e == cudaSuccess) return TP_OK;
    if (err) *err = std::string(what) + ": " + cudaGetErrorString(e);
    return TP_ERR_CUDA;
}

}  // namespace

namespace tpi {

int kv_write_launch(const PagedArgs& a, cudaStream_t stream, std::string* err) {
    if (a.n_seqs == 0) return TP_OK;
    const KvParams p = params_of(a);
    const long long groups = THREADS / (a.head_dim / 16);
    const long long need = (a.tokens * a.kv_heads + groups - 1) / groups;
    const dim3 grid(static_cast<unsigned>(std::min<long long>(need, device_sm_count() * 8LL))), block(THREADS);
    cudaError_t e;
    if (a.head_dim == 128)
        e = a.e4m3 ? launch_pdl(kv_write_kernel<128, true>, grid, block, 0, stream, p)
                   : launch_pdl(kv_write_kernel<128, false>, grid, block, 0, stream, p);
    else
        e = a.e4m3 ? launch_pdl(kv_write_kernel<64, true>, grid, block, 0, stream, p)
                   : launch_pdl(kv_write_kernel<64, false>, grid, block, 0, stream, p);
    return launched("cache write kernel", e, err);
}

int kv_read_launch(const PagedArgs& a, int64_t max_len, void* k_out, void* v_out, cudaStream_t stream,
                   std::string* err) {
    if (a.n_seqs == 0 || max_len == 0) return TP_OK;
    KvParams p = params_of(a);
    p.max_len = max_len;
    p.chunks = static_cast<int>((max_len + READ_POS - 1) / READ_POS);
    p.k_out = static_cast<__nv_bfloat16*>(k_out);
    p.v_out = static_cast<__nv_bfloat16*>(v_out);
    const long long blocks = static_cast<long long>(a.n_seqs) * p.chunks;
    if (blocks > 0x7fffffffll) {
        if (err) *err = "n_seqs x max_len is too large for one read";
        return TP_ERR_UNSUPPORTED;
    }
    const dim3 grid(static_cast<unsigned>(blocks)), block(THREADS);
    cudaError_t e;
    if (a.head_dim == 128)
        e = a.e4m3 ? launch_pdl(kv_read_kernel<128, true>, grid, block, 0, stream, p)
                   : launch_pdl(kv_read_kernel<128, false>, grid, block, 0, stream, p);
    else
        e = a.e4m3 ? launch_pdl(kv_read_kernel<64, true>, grid, block, 0, stream, p)
                   : launch_pdl(kv_read_kernel<64, false>, grid, block, 0, stream, p);
    return launched("cache read kernel", e, err);
}

}  // namespace tpi
