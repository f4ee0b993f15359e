// kv_attention_common.cuh -- what the two paged-attention kernels (kv_attention.cu, kv_attention_fp8.cu) share:
// the split of a context into parts, the launch's items and their distribution.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <atomic>

#include "kernels.h"
#include "ptx.cuh"

namespace dsa {
namespace kv {

// Parts of a context: of 2^kPartMin tokens, doubled until at most 2^parts_shift cover it.  All KV heads of one
// request make 128 parts, but at least 16 of a head: fewer leave SMs idle under one request, and every part costs
// its queries, its first base and its output beside its tiles.  128 is nowhere more than 1.2 times the best; 64 is
// up to 1.7 times it for one request, 256 costs the long batches.  Measured (4 KV heads of 128, calls in a row on the
// same inputs; their bytes in brackets):
//                                        64 parts   128 parts   256 parts
//   bf16, 1 x 128K (40 us)                 64.7        42.4        42.5 us
//   bf16, 4 x 32K (40)                     41.8        44.1        46.7
//   bf16, 24 x 8K (60)                     67.1        67.4        67.3
//   FP8, 1 x 128K (20)                     54.5        32.2        26.9
//   FP8, 24 x 8K (30)                      41.9        49.4        49.4
//   FP8, 32 x 16K-64K (203)               212         212         221
//   FP8, 4 x 4 rows of 60K-64K (38)        82.2        92.8       100
//   bf16, 23 ragged rows, 3 x 64           16.3        15.8        15.8
//   parts of at least                     128 tokens  256         512
//   bf16, one row of 4K                     9.4         9.5        11.0 us
//   FP8, 24 x 2K (7.6 us)                  24.6        19.8        20.0
//   FP8, 1 x 2K, 64 columns                12.2        13.3        17.1
constexpr int32_t kPartMin = 8;

__host__ __device__ __forceinline__ int32_t kv_parts_shift(int32_t kv_heads) {
    return kv_heads >= 8 ? 4 : kv_heads >= 4 ? 5 : kv_heads >= 2 ? 6 : 7;
}

// Bound of kv_parts over every context up to max_ctx.
inline uint32_t kv_parts_bound(int32_t max_ctx, int32_t parts_shift) {
    const int64_t n = (static_cast<int64_t>(max_ctx) + (1 << kPartMin) - 1) >> kPartMin, most = 1ll << parts_shift;
    return static_cast<uint32_t>(n < 1 ? 1 : (n < most ? n : most));
}

// log2 of a part's tokens: the smallest k >= part_min with 2^(k + parts_shift) >= ctx.
__device__ __forceinline__ int32_t kv_part_shift(int32_t ctx, int32_t parts_shift, int32_t part_min) {
    return part_min + (32 - __clz(max(ctx - 1, 0) >> (part_min + parts_shift)));
}

// A read, before the kernel's own griddepcontrol.wait, of what an earlier kernel wrote: the rows' lengths in the merges
// (kv_combine_kernel, kv_join_kernel); the split, the block table and the queries in kv_shared_kernel.  The writer was
// complete when the attention kernel in between passed its wait, and only then did that one let the next start, so the
// values are in L2.  But L1 may hold what a call before this one read at the same address (the same workspace in every
// layer, a block table that each step extends), and only the wait promises otherwise: so whatever is read before it is read
// past L1, by this, by cp.async.cg or by TMA.
template <typename T>
__device__ __forceinline__ T early_read(const T *p) {
    return __ldcg(p);
}

// An attention kernel works by itself, or beside kv_shared_kernel (where a.row_begin is there), with each row's first
// tokens left to that one.  kv_attention_kernel has a form for each: in one for both, 23 ragged rows of head_dim 64 take
// 16.7 us by themselves in the place of 16.4, four rows of 2K 8.8 and 8.5.  kv_attention_fp8_kernel has one for both: in
// forms of their own, 32 rows of 32K by themselves took 135.3 us in the place of 134.5, and what it tests stands at each
// branch, expected there (by way of a function, four groups of four rows of 64K took 97.5 us in the place of 91.3).
enum KvForm { kAlone, kBeside, kEither };

// What KvAttnArgs.row_begin says of a row: the first of its tokens that are read here, and log2 of its parts' least
// tokens below that (kPartMin or more).
constexpr int32_t kBeginUnit = 128;

template <int kForm>
__device__ __forceinline__ int32_t kv_begin(const KvAttnArgs &a, int row) {
    if (kForm == kEither ? __builtin_expect(a.row_begin == nullptr, 1) : kForm == kAlone) return kPartMin;
    return a.row_begin[row];
}
__device__ __forceinline__ int32_t kv_part_min(int32_t begin) { return begin & (kBeginUnit - 1); }

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

// ---- which items a CTA takes
//
// An item costs its tiles of 128 tokens and kItemCost more (its queries, its base, its output).  Counting items
// in the order (row group, KV head, column block, part), CTA b of n takes those that start within its n-th of the
// total cost: equal shares whatever the contexts (32 rows of 16K to 64K tokens: the busiest CTA has 1.09 times
// the mean; with items dealt in turn it had 1.28 to 1.44 times).  A share is one run of neighbours.
constexpr uint32_t kItemCost = 2;   // (3 and 4 measured the same)
constexpr int kMaxGroup = 8;        // rows of a group
constexpr int kSchedEntries = 512;  // running costs kept in shared memory, one for every so many groups

struct KvSchedule {
    int32_t mine, of;  // beside: this CTA's share (-1: none), and how many there are
    uint64_t before[kSchedEntries + 1];  // cost of all groups before the entry's
};

// Cost of a group with this longest context, for one KV head and column block.
__device__ __forceinline__ uint32_t kv_cost(int32_t ctx, int32_t part_shift) {
    return kv_parts(ctx, part_shift) * kItemCost + ((ctx + 127) >> 7);
}

__device__ __forceinline__ bool kv_direct(const KvAttnArgs &a) { return a.items <= gridDim.x; }  // an item a CTA

// Whether a row of context n and request req has no place in the group of a row of request first: its whole group is
// answered with nothing (out = 0, lse = -inf), as one part.
__device__ __forceinline__ bool kv_refused(const KvAttnArgs &a, int n, int req, int first) {
    return n < 0 || n > a.max_ctx || req != first || req < 0 || req >= a.num_requests;
}

// A lane's context of the group (of row `lane`, or of the first), its rows' request, and whether it is refused: then
// all contexts are 0.  Warp-collective.  kEarly: before the kernel's wait.
template <bool kEarly = false>
__device__ __forceinline__ int kv_load_group(const KvAttnArgs &a, int row0, int lane, int &req, bool &bad) {
    const int row = row0 + (lane < a.group ? lane : 0);
    const int n = kEarly ? early_read(a.row_ctx + row) : a.row_ctx[row];
    const int r = kEarly ? early_read(a.row_req + row) : a.row_req[row];
    req = __shfl_sync(0xffffffffu, r, 0);
    bad = __any_sync(0xffffffffu, kv_refused(a, n, r, req));
    return bad ? 0 : n;
}

// A row group's entries of the block table, from the first token that its rows read here.
__device__ __forceinline__ const int32_t *kv_table(const KvAttnArgs &a, int req, int32_t begin) {
    return a.block_table + static_cast<int64_t>(req) * a.bt_stride + ((begin & -kBeginUnit) >> a.page_shift);
}

// The share of a CTA where only own_sms[0] SMs are to work, two shares each: its SM's next one, if it has one left.  Where
// the SM has none (it is another kernel's, or CTAs of other SMs were quicker), the CTA takes a share of another SM while any
// is left; but the first two on an SM that is to have none leave at once.
// Those are at most 2 (gridDim / 2 - own_sms[0]) CTAs, however the CTAs are put and in whatever order they come.  All others,
// 2 own_sms[0] or more, end with a share or have seen that none is left: so none is left, and an atomic add gives each
// to one CTA.  Warp-collective; out of line, for the callers' registers.
[[maybe_unused]] static __device__ __noinline__ void kv_share(int32_t *own_sms, KvSchedule *sched, int lane) {
    int32_t *taken = own_sms + 1;  // by SM: its shares that are taken (more: nothing was left)
    uint32_t sm;
    asm volatile("mov.u32 %0, %%smid;" : "=r"(sm));
    int32_t v = 2;  // (both in one latency)
    if (lane == 0 && sm < kOwnSms) v = atomicAdd(taken + sm, 1);
    if (lane == 1) v = __ldcg(own_sms);
    const int n = __shfl_sync(0xffffffffu, v, 0), sms = __shfl_sync(0xffffffffu, v, 1);
    const uint32_t ctas = gridDim.x;
    int mine = static_cast<int>(blockIdx.x), of = static_cast<int>(ctas);
    if (2 * sms < of) {
        const bool one_of = sm < static_cast<uint32_t>(sms);
        of = 2 * sms;
        mine = one_of && n < 2 ? 2 * static_cast<int>(sm) + n : -1;
        // (an SM is found full once at most, so the bound never ends the search)
        const int most = mine >= 0 || (!one_of && n < 2 && sm < ctas / 2) ? 0 : sms + 1;
#pragma unroll 1
        for (int tries = 0; tries < most && mine < 0; ++tries) {
            int at = sms;  // of the SMs from one on that differs from CTA to CTA, the first with a share left
#pragma unroll 1
            for (int i = lane; i < sms && at == sms; i += 32)
                if (__ldcg(taken + (blockIdx.x + i) % sms) < 2) at = i;
            at = __reduce_min_sync(0xffffffffu, at);
            if (at == sms) break;
            const int from = static_cast<int>((blockIdx.x + at) % sms);
            const int m = __shfl_sync(0xffffffffu, lane == 0 ? atomicAdd(taken + from, 1) : 0, 0);
            if (m < 2) mine = 2 * from + m;
        }
    }
    if (lane == 0) {
        sched->mine = mine;
        sched->of = of;
    }
}

// Fills `sched`; every thread of the CTA calls it, then __syncthreads.  False: the CTA is to leave its SM to another kernel,
// at once, since that one waits for its place.
template <int kForm>
__device__ __forceinline__ bool kv_fill_schedule(const KvAttnArgs &a, KvSchedule *sched) {
    if (kv_direct(a)) return true;
    if (kForm == kEither ? __builtin_expect(a.own_sms != nullptr, 0) : kForm == kBeside) {
        if (threadIdx.x < 32) kv_share(a.own_sms, sched, threadIdx.x);
        __syncthreads();
        if (sched->mine < 0) return false;
    }
    const int per = a.sched_per, entries = a.sched_entries;
    for (int e = threadIdx.x; e < entries; e += blockDim.x) {
        uint64_t sum = 0;
#pragma unroll 1
        for (int gi = e * per; gi < min(a.groups, (e + 1) * per); ++gi) {
            // (all loads first: one latency)
            const int row0 = gi * a.group;
            int n[kMaxGroup], req[kMaxGroup];
            const int32_t begin = kv_begin<kForm>(a, row0);
#pragma unroll
            for (int r = 0; r < kMaxGroup; ++r) {
                const int row = row0 + (r < a.group ? r : 0);
                n[r] = a.row_ctx[row];
                req[r] = a.row_req[row];
            }
            bool bad = false;
            int ctx = 0;
#pragma unroll
            for (int r = 0; r < kMaxGroup; ++r) {
                bad |= kv_refused(a, n[r], req[r], req[0]);
                ctx = max(ctx, n[r]);
            }
            if (bad) ctx = 0;
            sum += kv_cost(ctx, kv_part_shift(ctx, a.parts_shift, kv_part_min(begin)));
        }
        sched->before[e + 1] = sum * (static_cast<uint64_t>(a.kv_heads) * a.col_blocks);
    }
    __syncthreads();
    if (threadIdx.x < 32) {
        const int lane = threadIdx.x;
        uint64_t carry = 0;
        if (lane == 0) sched->before[0] = 0;
#pragma unroll 1
        for (int e0 = 1; e0 <= entries; e0 += 32) {
            uint64_t v = e0 + lane <= entries ? sched->before[e0 + lane] : 0;
#pragma unroll 1
            for (int o = 1; o < 32; o <<= 1) {  // (rolled: code that runs once waits for its way in)
                const uint64_t u = __shfl_up_sync(0xffffffffu, v, o);
                if (lane >= o) v += u;
            }
            v += carry;
            if (e0 + lane <= entries) sched->before[e0 + lane] = v;
            carry = __shfl_sync(0xffffffffu, v, 31);
        }
    }
    return true;
}

// An item, and the way to the next one of this CTA.  Warp-collective.
template <int kForm>
struct KvCursor {
    int part, parts, col0, g, row0, req, t_begin, t_end, ctx, ctx_min;
    int my_ctx;  // of row `lane` of the group
    bool bad;
    int group, head, shift;  // head: KV head and column block
    int32_t begin;           // kv_begin
    uint64_t start, end;     // cost before the item, and where this CTA's share ends

    __device__ __forceinline__ void load_group(const KvAttnArgs &a, int lane) {
        row0 = group * a.group;
        begin = kv_begin<kForm>(a, row0);
        my_ctx = kv_load_group(a, row0, lane, req, bad);
        ctx = __reduce_max_sync(0xffffffffu, my_ctx);
        ctx_min = __reduce_min_sync(0xffffffffu, my_ctx);
        shift = kv_part_shift(ctx, a.parts_shift, kv_part_min(begin));
        parts = kv_parts(ctx, shift);
    }

    template <int kCols>
    __device__ __forceinline__ void place(const KvAttnArgs &a) {
        g = head;
        col0 = 0;
        if (a.col_blocks > 1) {
            g = static_cast<int>(static_cast<uint32_t>(head) / a.col_blocks);
            col0 = static_cast<int>(head - g * a.col_blocks) * kCols;
        }
        t_begin = part << shift;
        t_end = t_begin + min(ctx - t_begin, 1 << shift);
    }

    // The CTA's first item; false: it has none.
    template <int kCols>
    __device__ __forceinline__ bool first(const KvAttnArgs &a, const KvSchedule *sched, int lane) {
        const int heads = a.kv_heads * static_cast<int>(a.col_blocks);
        if (kv_direct(a)) {
            // (the numbers are small, so the halves keep the quotients clear of whole numbers)
            const int b = static_cast<int>(blockIdx.x), parts_of = static_cast<int>(a.parts_bound);
            const int j = static_cast<int>(__fdividef(b + 0.5f, static_cast<float>(parts_of)));
            part = b - j * parts_of;
            group = static_cast<int>(__fdividef(j + 0.5f, static_cast<float>(heads)));
            head = j - group * heads;
            start = end = 0;
            load_group(a, lane);
            place<kCols>(a);
            return part < parts;
        }
        const int per = a.sched_per, entries = a.sched_entries;
        // total * b / n: exact for products below 2^64 / n, and no total is near (a token costs 2^-6 or less)
        const uint64_t total = sched->before[entries];
        uint64_t from;
        if (kForm == kEither ? __builtin_expect(a.own_sms == nullptr, 1) : kForm == kAlone) {
            from = __umul64hi(total * blockIdx.x, a.ctas_inv);
            end = __umul64hi(total * (blockIdx.x + 1), a.ctas_inv);
        } else {
            from = total * sched->mine / sched->of;
            end = total * (sched->mine + 1) / sched->of;
        }
        if (from >= end) return false;
        int lo = 0;  // the last entry with nothing of the share before it
#pragma unroll 1
        for (int e = lane; e < entries; e += 32)
            if (sched->before[e] <= from) lo = e;
        lo = __reduce_max_sync(0xffffffffu, lo);
        start = sched->before[lo];
        group = lo * per;
        uint32_t unit;  // cost of a KV head and column block
#pragma unroll 1
        for (;; ++group) {
            load_group(a, lane);
            unit = kv_cost(ctx, shift);
            const uint64_t all = static_cast<uint64_t>(unit) * heads;
            if (start + all > from) break;
            start += all;
        }
        // the first item that starts at or past `from`
        uint64_t left = from - start;
        head = 0;
        if (left >= unit) {  // (the quotient is below heads, so fp32 misses it by one at most)
            head = static_cast<int>(__fdividef(__ull2float_rz(left), static_cast<float>(unit)));
            head -= static_cast<uint64_t>(head) * unit > left;
            head += static_cast<uint64_t>(head + 1) * unit <= left;
            left -= static_cast<uint64_t>(head) * unit;
        }
        start = from - left;
        const uint32_t step = kItemCost + (1u << (shift - 7));  // of every part but the last
        part = static_cast<int>(__fdividef(static_cast<float>(left), static_cast<float>(step)));  // (at most 128)
        while (static_cast<uint32_t>(part) * step < left) ++part;
        start += static_cast<uint64_t>(part) * step;
        if (part >= parts) {
            start = from - left + unit;
            part = parts - 1;
            return skip<kCols>(a, lane);
        }
        place<kCols>(a);
        return start < end;
    }

    // Step to the item after (group, head, part), which starts at `start`.
    template <int kCols>
    __device__ __forceinline__ bool skip(const KvAttnArgs &a, int lane) {
        if (start >= end) return false;
        if (++part >= parts) {
            part = 0;
            if (++head >= a.kv_heads * static_cast<int>(a.col_blocks)) {
                head = 0;
                ++group;
                load_group(a, lane);
            }
        }
        place<kCols>(a);
        return true;
    }

    template <int kCols>
    __device__ __forceinline__ bool next(const KvAttnArgs &a, int lane) {
        start += kItemCost + static_cast<uint32_t>((t_end - t_begin + 127) >> 7);
        return skip<kCols>(a, lane);
    }
};

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// A part's base as the merge takes it.  A part without any weight (a row of a group that ends before it, or scores
// that are all -inf) has none: 0 in its place would be the row's largest where all scores lie below, and the factors
// 2^(base - largest) of the parts that count would underflow.
__device__ __forceinline__ float part_base(float b, float sum) { return sum == 0.f ? -INFINITY : b; }

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
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

// Every lane asks, which orders the phase before every lane's later reads, and all go on together.
__device__ __forceinline__ bool wait_mbar_warp(uint64_t *bar, uint32_t parity, volatile int *abort) {
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
    const long long t0 = clock64();
#pragma unroll 1
    while (!__all_sync(0xffffffffu, mbar_try_wait(bar, parity)))
        if (__any_sync(0xffffffffu, *abort || clock64() - t0 > kWaitTimeoutCycles)) return false;
    return true;
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
inline uint32_t persistent_ctas(KvAttnArgs &a) {
    const uint32_t most = 2u * static_cast<uint32_t>(device_sm_count()), ctas = a.items < most ? a.items : most;
    if (ctas > 0) a.ctas_inv = ~0ull / ctas + 1;
    a.groups = a.num_rows / a.group;
    a.sched_per = (a.groups + kSchedEntries - 1) / kSchedEntries;
    a.sched_entries = (a.groups + a.sched_per - 1) / a.sched_per;
    return ctas;
}

}  // namespace kv
}  // namespace dsa
