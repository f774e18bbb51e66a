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
//
// One launch: a cluster of 8 CTAs per sequence, an eighth of the vocabulary
// each.  Up to 8 rows (16 rows of logits with the draft's) are summed at a
// time, every thread its pieces of one row after the other with a running
// maximum and loads in flight across rows; only the maxima and sums
// are exchanged, through distributed shared memory, as the vocabulary-parallel
// loss does between its shards.  Every CTA then decides by itself, and the race
// runs over the one row where a draft was refused (its logits are read a second
// time, from L2).  Bound by reading the logits once; rows behind a refused
// draft are still read if they are among its 8.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <string>

#include "tp_device.cuh"
#include "tp_internal.h"
#include "tp_packed.cuh"

namespace {

using namespace tpk;

constexpr int CS = 8;      // CTAs of a cluster
constexpr int WARPS = 8;   // small CTAs, four an SM: a batch of 64 sequences is one wave
constexpr int VT = WARPS * 32;
constexpr int ROWS = 8;    // rows of a batch
constexpr int FLY = 4;     // 16-byte loads in flight a thread
constexpr float LOG2E = 1.4426950408889634f;

struct VerifyParams {
    const __nv_bfloat16 *z, *y;
    long long rows, v;
    const int32_t *ids, *q_start;
    const float *temperature, *u, *noise;
    int32_t *accepted, *tokens;
};

__device__ __forceinline__ float ex2f(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// m = max x_v and s = sum 2^((x_v - m) it), it = log2(e) / T.
struct Stat {
    float m, s;
};
__device__ __forceinline__ Stat merge(Stat a, Stat b, float it) {
    const float m = fmaxf(a.m, b.m);
    if (m == -INFINITY) return {m, 0.0f};
    return {m, a.s * ex2f((a.m - m) * it) + b.s * ex2f((b.m - m) * it)};
}

// Largest value and its lowest index.
struct Best {
    float v;
    int i;
};
__device__ __forceinline__ Best better(Best a, Best b) {
    return (b.v > a.v || (b.v == a.v && b.i < a.i)) ? b : a;
}
__device__ __forceinline__ Best warp_best(Best a) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const Best b = {__shfl_xor_sync(0xffffffffu, a.v, o), __shfl_xor_sync(0xffffffffu, a.i, o)};
        a = better(a, b);
    }
    return a;
}

// 8 bytes to the same shared-memory address in CTA `rank` of the cluster.
__device__ __forceinline__ void store_cluster(uint32_t addr, int rank, uint32_t a, uint32_t b) {
    asm volatile("st.shared::cluster.v2.b32 [%0], {%1, %2};" ::"r"(mapa_shared(addr, static_cast<uint32_t>(rank))), "r"(a),
                 "r"(b)
                 : "memory");
}

__device__ __forceinline__ float prob(float x, float it, Stat st) {
    return st.s > 0.0f ? ex2f((x - st.m) * it) / st.s : 0.0f;
}

__global__ void __cluster_dims__(CS, 1, 1) __launch_bounds__(VT, 4) verify_kernel(const VerifyParams p) {
    pdl_trigger();
    pdl_wait();
    __shared__ Stat part[2 * ROWS][VT];    // by row of logits: a thread's statistics, or its largest logit
    __shared__ Stat all[2][2 * ROWS][CS];  // by batch parity, row of logits and CTA
    __shared__ Best race[WARPS][2], raced[CS][2];
    const int rank = static_cast<int>(cluster_ctarank()), warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int s = blockIdx.x / CS;
    const long long r0 = min(max(static_cast<long long>(p.q_start[s]), 0ll), p.rows);
    const long long r1 = min(max(static_cast<long long>(p.q_start[s + 1]), r0), p.rows);
    const int n = static_cast<int>(r1 - r0);
    if (n == 0) {  // the whole cluster
        if (rank == 0 && threadIdx.x == 0) p.accepted[s] = 0;
        return;
    }
    const float T = p.temperature ? p.temperature[s] : 1.0f;
    const bool greedy = !(T > 0.0f);
    const float it = fminf(LOG2E / T, 1e30f);  // finite, so that 0 * it is 0
    const int pieces = static_cast<int>(p.v / 8), mine = (pieces + CS - 1) / CS;
    const int begin = min(rank * mine, pieces), end = min(begin + mine, pieces);

    int taken = n - 1, token = -1;
    Stat sp = {-INFINITY, 0.0f}, sq = {-INFINITY, 0.0f};
    bool drafted = false;  // the row that stops has a draft distribution
    for (int b0 = 0, parity = 0; b0 < n; b0 += ROWS, parity ^= 1) {
        const int rows = min(ROWS, n - b0);
        // Rows of logits: the target's, then the draft's (none behind the last draft).
        const int drafts = greedy || !p.y ? 0 : min(rows, n - 1 - b0);
        const int items = rows + drafts;
        // Pieces of 8 logits (16 bytes): this thread's of a row are begin + threadIdx.x + j VT; one row after the
        // other, FLY loads in flight.
        const int turns = (end - begin + VT - 1) / VT;
        auto row_of = [&](int i) {
            return reinterpret_cast<const uint4*>(i < rows ? p.z + (r0 + b0 + i) * p.v : p.y + (r0 + b0 + i - rows) * p.v);
        };
        Stat a = {-INFINITY, 0.0f};
        int li = 0, lj = 0;  // row and piece of the next load
        int ui = 0, uj = 0;  // and of the next use
        const int first = begin + static_cast<int>(threadIdx.x);
        for (int k0 = 0; k0 < items * turns; k0 += FLY) {
            uint4 u[FLY];
#pragma unroll
            for (int e = 0; e < FLY; ++e) {
                if (li < items && first + lj * VT < end) u[e] = row_of(li)[first + lj * VT];
                if (++lj == turns) {
                    lj = 0;
                    ++li;
                }
            }
#pragma unroll
            for (int e = 0; e < FLY; ++e) {
                if (ui == items) break;
                const int piece = first + uj * VT;
                if (piece < end) {
                    const uint32_t w[4] = {u[e].x, u[e].y, u[e].z, u[e].w};
                    float v[8];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const float2 t = unpack_bf16x2(w[k]);
                        v[2 * k] = t.x;
                        v[2 * k + 1] = t.y;
                    }
                    if (greedy) {
#pragma unroll
                        for (int k = 0; k < 8; ++k)
                            if (v[k] > a.m) a = {v[k], __int_as_float(piece * 8 + k)};  // indices ascend in a thread
                    } else {
                        const float bm = max3(max3(v[0], v[1], v[2]), max3(v[3], v[4], v[5]), fmaxf(v[6], v[7]));
                        if (bm > a.m) {
                            a.s *= ex2f((a.m - bm) * it);  // 0 * 0 at first
                            a.m = bm;
                        }
                        if (a.m > -INFINITY) {
                            // The difference first, as everywhere: exact for near logits, finite at the type's ends.
                            const uint64_t minus = f2_pack(-a.m, -a.m), its = f2_pack(it, it);
                            float x[8];
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                float x0, x1;
                                f2_unpack(f2_mul(f2_add(f2_pack(v[2 * k], v[2 * k + 1]), minus), its), x0, x1);
                                x[2 * k] = ex2f(x0);
                                x[2 * k + 1] = ex2f(x1);
                            }
                            a.s += ((x[0] + x[1]) + (x[2] + x[3])) + ((x[4] + x[5]) + (x[6] + x[7]));
                        }
                    }
                }
                if (++uj == turns) {
                    part[ui][threadIdx.x] = a;
                    a = {-INFINITY, 0.0f};
                    uj = 0;
                    ++ui;
                }
            }
        }
        __syncthreads();
        // A warp a row: the CTA's statistics, to every CTA of the cluster.
        for (int i = warp; i < items; i += WARPS) {
            Stat b = {-INFINITY, 0.0f};
            if (turns > 0) b = part[i][lane];
            if (greedy) {
                Best c = {b.m, b.m > -INFINITY ? __float_as_int(b.s) : 0x7fffffff};
                for (int k = 32; turns > 0 && k < VT; k += 32) {
                    const Stat d = part[i][lane + k];
                    if (d.m > -INFINITY) c = better(c, {d.m, __float_as_int(d.s)});
                }
                c = warp_best(c);
                b = {c.v, __int_as_float(c.i)};
            } else {
                for (int k = 32; turns > 0 && k < VT; k += 32) b = merge(b, part[i][lane + k], it);
#pragma unroll
                for (int o = 16; o > 0; o >>= 1)
                    b = merge(b, {__shfl_xor_sync(0xffffffffu, b.m, o), __shfl_xor_sync(0xffffffffu, b.s, o)}, it);
            }
            if (lane < CS)
                store_cluster(smem_u32(&all[parity][i][rank]), lane, __float_as_uint(b.m), __float_as_uint(b.s));
        }
        // A batch's buffer is written again two batches on: behind the next batch's barrier, which every CTA
        // reaches after it has read this one.
        cluster_sync_all();
        // Every warp decides, a lane a row.
        bool take = false;
        Stat tp_ = {-INFINITY, 0.0f}, tq = {-INFINITY, 0.0f};
        if (lane < rows) {
            const long long r = r0 + b0 + lane;
            const bool last = b0 + lane + 1 == n;
            const long long x = last ? -1 : p.ids[r + 1];
            const bool inside = x >= 0 && x < p.v;
            tp_ = all[parity][lane][0];
            for (int k = 1; k < CS; ++k) {
                const Stat b = all[parity][lane][k];
                if (greedy) {
                    const Best c = better({tp_.m, __float_as_int(tp_.s)}, {b.m, __float_as_int(b.s)});
                    tp_ = {c.v, __int_as_float(c.i)};
                } else {
                    tp_ = merge(tp_, b, it);
                }
            }
            if (greedy) {
                take = inside && tp_.m > -INFINITY && __float_as_int(tp_.s) == static_cast<int>(x);
            } else {
                if (lane < drafts) {
                    tq = all[parity][rows + lane][0];
                    for (int k = 1; k < CS; ++k) tq = merge(tq, all[parity][rows + lane][k], it);
                }
                if (inside) {
                    const float px = prob(__bfloat162float(p.z[r * p.v + x]), it, tp_);
                    const float qx = lane < drafts ? prob(__bfloat162float(p.y[r * p.v + x]), it, tq) : 0.0f;
                    take = p.u[r] * qx < px;
                }
            }
        }
        const unsigned kept = __ballot_sync(0xffffffffu, lane < rows && !take);
        if (kept) {
            const int i = __ffs(kept) - 1;
            taken = b0 + i;
            sp = {__shfl_sync(0xffffffffu, tp_.m, i), __shfl_sync(0xffffffffu, tp_.s, i)};
            sq = {__shfl_sync(0xffffffffu, tq.m, i), __shfl_sync(0xffffffffu, tq.s, i)};
            drafted = i < drafts;
            break;
        }
    }
    if (greedy) {
        token = sp.m > -INFINITY ? __float_as_int(sp.s) : -1;
    } else {
        // The race over w = max(0, p - q), and over p alone in case that leaves nothing.
        Best b = {0.0f, 0x7fffffff}, f = b;
        const uint4* z = reinterpret_cast<const uint4*>(p.z + (r0 + taken) * p.v);
        const uint4* y = drafted ? reinterpret_cast<const uint4*>(p.y + (r0 + taken) * p.v) : nullptr;
        const float4* e4 = p.noise ? reinterpret_cast<const float4*>(p.noise + s * p.v) : nullptr;
        const float ip = sp.s > 0.0f ? 1.0f / sp.s : 0.0f, iq = sq.s > 0.0f ? 1.0f / sq.s : 0.0f;
#pragma unroll 2
        for (int c = begin + static_cast<int>(threadIdx.x); c < end; c += VT) {
            const uint4 zu = z[c], yu = y ? y[c] : make_uint4(0, 0, 0, 0);
            const float4 one = make_float4(1.0f, 1.0f, 1.0f, 1.0f);
            const float4 ea = e4 ? __ldcs(e4 + 2 * c) : one, eb = e4 ? __ldcs(e4 + 2 * c + 1) : one;
            const uint32_t zw[4] = {zu.x, zu.y, zu.z, zu.w}, yw[4] = {yu.x, yu.y, yu.z, yu.w};
            const float e[8] = {ea.x, ea.y, ea.z, ea.w, eb.x, eb.y, eb.z, eb.w};
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const float2 zf = unpack_bf16x2(zw[k >> 1]), yf = unpack_bf16x2(yw[k >> 1]);
                const float pv = ex2f((((k & 1) ? zf.y : zf.x) - sp.m) * it) * ip;
                const float qv = y ? ex2f((((k & 1) ? yf.y : yf.x) - sq.m) * it) * iq : 0.0f;
                // A probability of NaN, as from NaN or infinite logits, wins nothing.
                const float rb = __fdividef(pv - (iq > 0.0f ? qv : 0.0f), e[k]), rf = __fdividef(pv, e[k]);
                if (rb > b.v) b = {rb, c * 8 + k};
                if (rf > f.v) f = {rf, c * 8 + k};
            }
        }
        b = warp_best(b);
        f = warp_best(f);
        if (lane == 0) {
            race[warp][0] = b;
            race[warp][1] = f;
        }
        __syncthreads();
        if (threadIdx.x < 2) {
            Best a = race[0][threadIdx.x];
            for (int k = 1; k < WARPS; ++k) a = better(a, race[k][threadIdx.x]);
            store_cluster(smem_u32(&raced[rank][threadIdx.x]), 0, __float_as_uint(a.v), static_cast<uint32_t>(a.i));
        }
        cluster_sync_all();
        if (rank == 0) {
            b = raced[0][0];
            f = raced[0][1];
            for (int k = 1; k < CS; ++k) {
                b = better(b, raced[k][0]);
                f = better(f, raced[k][1]);
            }
            if (!(b.v > 0.0f)) b = f;
            token = b.v > 0.0f ? b.i : -1;
        }
    }
    if (rank == 0) {
        if (threadIdx.x == 0) p.accepted[s] = taken;
        for (int i = threadIdx.x; i < n; i += VT)
            p.tokens[r0 + i] = i < taken ? p.ids[r0 + i + 1] : i == taken ? token : -1;
    }
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
    cudaError_t e = launch_pdl(verify_kernel, dim3(static_cast<unsigned>(a.n_seqs) * CS), dim3(VT), 0, stream, p);
    if (e == cudaSuccess) e = cudaGetLastError();
    if (e != cudaSuccess) {
        if (err) *err = std::string("verification kernel: ") + cudaGetErrorString(e);
        return TP_ERR_CUDA;
    }
    return TP_OK;
}

}  // namespace tpi
