// tp_attn_paged.cuh -- what the two kernels of attention over a paged cache
// share: a CTA's share of the work, the cache's tensor maps, and the scratch of
// split tiles.
#pragma once

#include <cuda.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <string>

#include "tp_device.cuh"
#include "tp_internal.h"
#include "tp_paged.cuh"

namespace tpk {

// 2^x (PTX ex2.approx.ftz: relative error about 2^-22, -inf -> +0).
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int32_t c0, int32_t c1,
                                            int32_t c2, int32_t c3) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
        : "memory");
}

// Bring a box of a tensor map into L2.
__device__ __forceinline__ void tma_prefetch_l2_4d(const CUtensorMap* map, int32_t c0, int32_t c1, int32_t c2, int32_t c3) {
    asm volatile("cp.async.bulk.prefetch.tensor.4d.L2.global.tile [%0, {%1, %2, %3, %4}];" ::"l"(
                     reinterpret_cast<uint64_t>(map)),
                 "r"(c0), "r"(c1), "r"(c2), "r"(c3)
                 : "memory");
}

__device__ __forceinline__ float ld_shared_f32(uint32_t addr) {
    float v;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}

// Two e4m3 codes (low 16 bits), exactly; NaN stays NaN.
__device__ __forceinline__ uint32_t e4m3x2_f16x2(uint32_t codes) {
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<uint16_t>(codes)));
    return r;
}
__device__ __forceinline__ float2 e4m3x2_float2(uint32_t codes) {
    const uint32_t h = e4m3x2_f16x2(codes);
    return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// 16 bytes to shared memory by this thread, and its arrival at a barrier once all such copies of its own are there
// (the barrier counts that arrival from the start).
__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copies_arrive(uint32_t bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// Contiguous copy to shared memory; addresses and size multiples of 16 bytes.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "l"(src), "r"(bytes), "r"(bar)
                 : "memory");
}

// mbar_wait with its loop out of line: the waits of a kernel's roles, inlined
// with it, took more of the instruction cache than the work between them.
__device__ __noinline__ inline bool bar_wait_slow(uint32_t bar, uint32_t parity, volatile int* abort_flag, unsigned* status,
                                                  uint64_t timeout_ns) {
    return mbar_wait(bar, parity, abort_flag, status, timeout_ns);
}
struct Waiter {
    volatile int* abort_flag;
    unsigned* status;
    uint64_t timeout_ns;
    __device__ __forceinline__ bool operator()(uint32_t bar, uint32_t parity) const {
        return mbar_try_wait(bar, parity) || bar_wait_slow(bar, parity, abort_flag, status, timeout_ns);
    }
};

// total / grid rounded up, without a 64-bit division: an approximate quotient,
// corrected by the remainder (below 2^31 for total < 2^50).
__device__ __forceinline__ long long share_size(long long total, int grid) {
    const long long q = static_cast<long long>(__ll2float_rn(total) / static_cast<float>(grid));
    const int rem = static_cast<int>(total - q * grid);
    const int more = rem >= 0 ? (rem + grid - 1) / grid : -(-rem / grid);
    return q + more;
}

// The CTA whose share holds block `at`: at / per, the same way.
__device__ __forceinline__ int share_of(long long at, long long per) {
    long long q = static_cast<long long>(__ll2float_rn(at) / __ll2float_rn(per));
    while (q * per > at) --q;
    while ((q + 1) * per <= at) ++q;
    return static_cast<int>(q);
}

// The share of CTA blockIdx.x: its first block, their number, every CTA's
// number; walk gets its beginning.  Called by every warp (walk: its own, in
// shared memory).  Sequences are summed in runs, and a scan of the sums finds
// the one where the share begins; the tile is then looked for 32 at a time.  Up
// to 256 sequences every warp does that alone, a run a lane: two barriers of
// the CTA less in front of its first load.  More: a run a thread.  What a lane
// found of its sequence goes to the others by shuffles: a second read of its
// lengths, and a second count of its blocks, cost about 2000 cycles.  sums: NT /
// 32 + 2 words of 8 bytes of shared memory.
struct Share {
    long long begin, count, per;
};
template <int NT>
__device__ __forceinline__ Share find_share(const PagedView& v, const Tiling& t, long long* sums, TileWalk& walk) {
    const int tid = threadIdx.x, lane = tid & 31;
    const bool alone = v.n_seqs <= 256;
    const int run = alone ? (v.n_seqs + 31) / 32 : (v.n_seqs + NT - 1) / NT;
    const int s0 = min((alone ? lane : tid) * run, v.n_seqs), s1 = min(s0 + run, v.n_seqs);
    long long mine = 0, per_head = 0;
    PagedSeq q = {0, 0, 0};
#pragma unroll 1
    for (int s = s0; s < s1; ++s) {
        q = paged_seq(v, s);
        per_head = head_blocks(v, q, t);
        mine += per_head * v.kv_heads;
    }
    long long inc = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long x = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += x;
    }
    long long before = inc - mine, total = __shfl_sync(0xffffffffu, inc, 31);
    if (__builtin_expect(!alone, 0)) {
        if (lane == 31) sums[tid >> 5] = inc;
        __syncthreads();
        total = 0;
#pragma unroll 1
        for (int w = 0; w < NT / 32; ++w) {
            if (w < (tid >> 5)) before += sums[w];
            total += sums[w];
        }
    }
    Share x;
    x.per = share_size(total, static_cast<int>(gridDim.x));
    x.begin = pmin(static_cast<long long>(blockIdx.x) * x.per, total);
    x.count = pmin(x.per, total - x.begin);
    const bool here = x.count > 0 && x.begin >= before && x.begin < before + mine;
    int s = s0;
    long long off = x.begin - before;
    if (__builtin_expect(run > 1 && here, 0)) {
#pragma unroll 1
        for (;; ++s) {
            q = paged_seq(v, s);
            per_head = head_blocks(v, q, t);
            if (s == s1 - 1 || off < per_head * v.kv_heads) break;
            off -= per_head * v.kv_heads;
        }
    }
    if (__builtin_expect(alone, 1)) {
        const unsigned who = __ballot_sync(0xffffffffu, here);
        const int from = who ? __ffs(who) - 1 : 0;
        s = __shfl_sync(0xffffffffu, s, from);
        off = __shfl_sync(0xffffffffu, off, from);
        per_head = __shfl_sync(0xffffffffu, per_head, from);
        q.row0 = __shfl_sync(0xffffffffu, q.row0, from);
        q.n = __shfl_sync(0xffffffffu, q.n, from);
        q.len = __shfl_sync(0xffffffffu, q.len, from);
    } else {
        if (here) {
            sums[NT / 32] = off;
            sums[NT / 32 + 1] = s;
        }
        __syncthreads();
        off = sums[NT / 32];
        s = static_cast<int>(sums[NT / 32 + 1]);
        if (x.count > 0) {
            q = paged_seq(v, s);
            per_head = head_blocks(v, q, t);
        }
    }
    if (x.count > 0) {
        const int keys = paged_keys(v, q), tiles = seq_tiles(q, t);
        int g = 0;
#pragma unroll 1
        for (; off >= per_head; ++g) off -= per_head;
        // The last tile that begins at or before `off`: of [lo, lo + 32 step) by its 32 steps, then within one.
        int lo = 0, step = 1;
        if (tiles > 1) {
            while (step * 32 < tiles) step *= 32;
#pragma unroll 1
            for (;; step /= 32) {
                const int at = lo + lane * step;
                const long long blocks = tiles_blocks(q, keys, t, at < tiles ? at : 0);
                const int last = __popc(__ballot_sync(0xffffffffu, at < tiles && blocks <= off)) - 1;
                lo += last * step;
                if (step == 1) {
                    off -= __shfl_sync(0xffffffffu, blocks, last);
                    break;
                }
            }
        }
        if (lane == 0) {
            walk.q = q;
            walk.left = x.count;
            walk.s = s;
            walk.g = g;
            walk.tile = lo;
            walk.tiles = tiles;
            walk.keys = keys;
            walk.kb = static_cast<int>(off);
            walk.nkb = tile_blocks(q, keys, t, lo);
        }
    } else if (lane == 0) {
        walk.left = 0;
    }
    __syncwarp();
    return x;
}

// Wait for copies in flight when a role gives up.
__device__ __forceinline__ void drain(uint32_t bar, uint32_t parity) {
    const uint64_t t0 = globaltimer_ns();
    while (!mbar_try_wait(bar, parity))
        if (globaltimer_ns() - t0 > 200000000ull) break;  // 200 ms
}

}  // namespace tpk

namespace tpi {

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

inline EncodeTiledFn find_encode_fn() {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult qr;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &qr) != cudaSuccess ||
        qr != cudaDriverEntryPointSuccess)
        return nullptr;
    return reinterpret_cast<EncodeTiledFn>(f);
}
// The driver's entry point, looked up once a process.
inline EncodeTiledFn encode_fn(std::string* err) {
    static const EncodeTiledFn found = find_encode_fn();
    if (!found && err) *err = "cuTensorMapEncodeTiled is not available from the driver";
    return found;
}

// The cache as {d, page, k, n_pages} with boxes of `span` bytes of a row (swizzled over that span) by box_rows;
// span 0: whole rows, as they are.
inline int encode_cache(CUtensorMap* map, const PagedArgs& a, const void* base, int span, int box_rows, std::string* err) {
    EncodeTiledFn encode = encode_fn(err);
    if (!encode) return TP_ERR_CUDA;
    const cuuint64_t elem = a.e4m3 ? 1 : 2;
    const cuuint64_t d = static_cast<cuuint64_t>(a.head_dim), pg = static_cast<cuuint64_t>(a.page_size);
    const cuuint64_t dims[4] = {d, pg, static_cast<cuuint64_t>(a.kv_heads), static_cast<cuuint64_t>(a.n_pages)};
    const cuuint64_t strides[3] = {d * elem, d * pg * elem, d * pg * a.kv_heads * elem};
    const cuuint32_t box[4] = {static_cast<cuuint32_t>(span ? span / elem : d), static_cast<cuuint32_t>(box_rows), 1, 1};
    const cuuint32_t estr[4] = {1, 1, 1, 1};
    const CUresult r = encode(map, a.e4m3 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4,
                              const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                              span == 0    ? CU_TENSOR_MAP_SWIZZLE_NONE
                              : span == 128 ? CU_TENSOR_MAP_SWIZZLE_128B
                                            : CU_TENSOR_MAP_SWIZZLE_64B,
                              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) {
        if (err) *err = "cuTensorMapEncodeTiled (cache) failed: " + std::to_string(static_cast<int>(r));
        return TP_ERR_CUDA;
    }
    return TP_OK;
}

inline int launched(const char* what, cudaError_t e, std::string* err) {
    if (e == cudaSuccess) e = cudaGetLastError();
    if (e == cudaSuccess) return TP_OK;
    if (err) *err = std::string(what) + ": " + cudaGetErrorString(e);
    return TP_ERR_CUDA;
}

// Scratch of a launch: partial results of `rows` x D, their statistics, descriptors.
struct Scratch {
    size_t o, ml, desc, total;
};
inline Scratch scratch_of(int grid, int rows, int D) {
    Scratch s;
    s.o = 0;
    s.ml = s.o + static_cast<size_t>(grid) * 2 * rows * D * 4;
    s.desc = s.ml + static_cast<size_t>(grid) * 2 * rows * 2 * 4;
    s.total = s.desc + static_cast<size_t>(grid) * 16;
    return s;
}

// Attention of many rows a sequence (tp_attn_chunk.cu), and the joining of the
// tiles that its shares, or those of the kernel for few rows, cut.
int attn_chunk_launch(const PagedArgs& a, void* O, void* scratch, bool zero_rest, cudaStream_t stream, std::string* err);
int attn_join_launch(const PagedArgs& a, int slot_rows, void* O, uint8_t* scratch, const Scratch& s, int grid,
                     bool zero_rest, cudaStream_t stream, std::string* err);

}  // namespace tpi
