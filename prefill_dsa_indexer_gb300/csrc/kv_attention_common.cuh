// kv_attention_common.cuh -- what the two paged-attention kernels (kv_attention.cu, kv_attention_fp8.cu) share:
// the split of a context into parts, the launch's items and their decoding.
#pragma once

#include <cuda_bf16.h>

#include <atomic>

#include "kernels.h"
#include "ptx.cuh"

namespace dsa {
namespace kv {

// Parts of a context: of 128 tokens, doubled until at most 2^parts_shift cover it.  parts_shift: 128 parts
// over all KV heads, so that one request alone gives most of the 152 SMs a CTA, but at least 16.
__host__ __device__ __forceinline__ int32_t kv_parts_shift(int32_t kv_heads) {
    return kv_heads >= 8 ? 4 : kv_heads >= 4 ? 5 : kv_heads >= 2 ? 6 : 7;
}

// log2 of a part's tokens: the smallest k >= 7 with 2^(k + parts_shift) >= ctx.
__device__ __forceinline__ int32_t kv_part_shift(int32_t ctx, int32_t parts_shift) {
    return 7 + (32 - __clz(max(ctx - 1, 0) >> (7 + parts_shift)));
}

__device__ __forceinline__ int32_t kv_parts(int32_t ctx, int32_t part_shift) {
    return max(1, (ctx + (1 << part_shift) - 1) >> part_shift);
}

// What the query warp tells the consumers about an item.
struct KvItem {
    int32_t live;       // 0: no more items
    int32_t t_begin, t_end;
    int32_t ctx_min;    // tokens that every row of the group sees
    int32_t row0, g, part, parts;
    int32_t ctx[8];     // the group's contexts
};
static_assert(sizeof(KvItem) == 64, "item layout");

// Item `i` of the launch: part fastest, then column block, KV head, row group.  Warp-collective; false:
// the group's context has fewer parts.
struct KvWhere {
    int part, parts, col0, g, row0, req, t_begin, t_end, ctx, ctx_min, my_ctx;
    bool bad;
};

template <int kCols>
__device__ __forceinline__ bool kv_where(const KvAttnArgs &a, uint32_t i, int lane, KvWhere &w) {
    uint32_t j = i / a.parts_bound;
    w.part = static_cast<int>(i - j * a.parts_bound);
    w.col0 = 0;
    if (a.col_blocks > 1) {
        const uint32_t k = j / a.col_blocks;
        w.col0 = static_cast<int>(j - k * a.col_blocks) * kCols;
        j = k;
    }
    const uint32_t k = j / a.kv_heads;
    w.g = static_cast<int>(j - k * a.kv_heads);
    w.row0 = static_cast<int>(k) * a.group;
    const int row = w.row0 + (lane < a.group ? lane : 0);
    const int n = a.row_ctx[row], req = a.row_req[row];
    w.req = __shfl_sync(0xffffffffu, req, 0);
    w.bad = __any_sync(0xffffffffu, n < 0 || n > a.max_ctx || req != w.req) || w.req < 0 || w.req >= a.num_requests;
    w.my_ctx = w.bad ? 0 : n;  // of row `lane` of the group
    w.ctx = __reduce_max_sync(0xffffffffu, w.my_ctx);
    w.ctx_min = __reduce_min_sync(0xffffffffu, w.my_ctx);
    const int shift = kv_part_shift(w.ctx, a.parts_shift);
    w.parts = kv_parts(w.ctx, shift);
    if (w.part >= w.parts) return false;
    w.t_begin = w.part << shift;
    w.t_end = w.t_begin + min(w.ctx - w.t_begin, 1 << shift);
    return true;
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}

__device__ __forceinline__ float bf16_lo(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t v) { return __uint_as_float(v & 0xffff0000u); }

// mbar_wait without the report, in few instructions: these kernels wait in twenty places, and code that does not
// stay in the instruction caches is slow to fetch beside the streamed data.  A role whose wait returned false
// calls gave_up, which makes the CTA's other waits return too.
__device__ __forceinline__ bool wait_mbar(uint64_t *bar, uint32_t parity, volatile int *abort) {
    if (mbar_try_wait(bar, parity)) return true;
    const long long t0 = clock64();
#pragma unroll 1
    while (!mbar_try_wait(bar, parity))
        if (*abort || clock64() - t0 > kWaitTimeoutCycles) return false;
    return true;
}

__device__ __forceinline__ bool wait_mbar_warp(uint64_t *bar, uint32_t parity, volatile int *abort) {
    int ok = 0;
    if ((threadIdx.x & 31) == 0) ok = wait_mbar(bar, parity, abort);
    ok = __shfl_sync(0xffffffffu, ok, 0);
    __syncwarp();  // orders lane 0's acquire before every lane's later reads
    return ok != 0;
}

__device__ __forceinline__ void gave_up(volatile int *abort, int32_t *status) {
    if (!*abort) report(status, DSA_ERR_TIMEOUT);
    *abort = 1;
}

// Raise `kern`'s shared-memory limit on the current device, once per device (`configured`: a bit each).
template <typename K>
inline cudaError_t raise_smem_limit(K kern, int bytes, std::atomic<uint64_t> &configured) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = 1ull << (dev & 63);
    if (dev < 64 && (configured.load() & bit)) return cudaSuccess;
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess && dev < 64) configured.fetch_or(bit);
    return e;
}

// CTAs of a persistent launch over a.items items, two per SM; 0: no device.
inline uint32_t persistent_ctas(const KvAttnArgs &a) {
    const uint32_t ctas = 2u * static_cast<uint32_t>(device_sm_count());
    return a.items < ctas ? a.items : ctas;
}

}  // namespace kv
}  // namespace dsa
