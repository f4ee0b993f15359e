// plan.cu -- the rows, slots and pages of a step of requests, from their lengths (dsa_kv_plan).
//
//   need_i = ceil((ctx_i + n_i) / page) - ceil(ctx_i / page)       pages that request i begins
//   rows_i = n_i, raised to a multiple of the rows per group
//   A_i = sum_{j <= i} need_j, B_i = sum_{j <= i} rows_j           request i gets its tokens if A_i and B_i fit
//   page k of request i's new ones is the (A_i - need_i + k)-th from the top of the stack of free pages
//   slot of position p = table[i][p / page] * page + p % page
//
// Sums over the requests and then four numbers a row: a few hundred KB for the largest steps, so nothing but latency
// counts, and it is one launch.  Every CTA of one cluster makes the same sums over all requests (lengths are few) and
// keeps them in shared memory; rows, pages begun and pages given back are shared out one by one, and each finds its
// request there by bisection.  (A warp a request for the pages: 27 us where 28 of 257 requests gave back 500 pages each.)
// What one CTA writes and another reads (pages given back) or what a call may update in place (contexts, the stack's
// count, which all CTAs read first) is set apart by cluster barriers.
#include <atomic>

#include "kernels.h"
#include "ptx.cuh"

namespace dsa {

namespace {

// A cluster of the largest portable size: one CTA takes as long for 8 rows (4.7 us in a graph), and 32 us in the place of
// 12 for 2,048 requests of 16,384 rows.
constexpr int kThreads = 1024, kWarps = kThreads / 32, kCtas = 8;
constexpr int kAtOnce = 8;  // pages given back that a thread has on their way

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}

// All threads of the cluster; what they wrote before is visible after.
__device__ __forceinline__ void cluster_meet() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// A request's lengths, checked.
struct Request {
    int32_t ctx, fresh;  // tokens in the cache, new ones
    int32_t had, need;   // pages listed, pages to begin
    int32_t back;        // pages to give back
    uint32_t wide;       // rows
    bool ended, bad;
};

__device__ __forceinline__ Request read_request(const KvPlanArgs &a, int i) {
    Request r = {};
    r.ctx = a.context[i];
    const int32_t n = a.new_tokens[i];
    const int32_t own = a.first_own != nullptr ? a.first_own[i] : 0;
    r.ended = n == -1;
    r.bad = r.ctx < 0 || r.ctx > a.capacity || n < -1 || n > a.capacity - r.ctx || own < 0;
    if (r.bad) return r;
    const auto pages = [&](int32_t t) { return static_cast<int32_t>((static_cast<uint32_t>(t) + a.page_size - 1) >> a.page_shift); };
    r.had = pages(r.ctx);
    if (r.ended) {
        r.back = max(r.had - own, 0);
    } else {
        r.fresh = n;
        r.need = pages(r.ctx + n) - r.had;
        r.wide = (static_cast<uint32_t>(n) + a.group - 1) / a.group * a.group;
    }
    return r;
}

struct Sums {
    int64_t need, wide, back;
    __device__ __forceinline__ void add(const Sums &o) {
        need += o.need;
        wide += o.wide;
        back += o.back;
    }
};

__device__ __forceinline__ Sums shifted(const Sums &s, int by) {
    return {__shfl_up_sync(0xffffffffu, s.need, by), __shfl_up_sync(0xffffffffu, s.wide, by),
            __shfl_up_sync(0xffffffffu, s.back, by)};
}

__device__ __forceinline__ int32_t capped(int64_t x) { return static_cast<int32_t>(x < INT32_MAX ? x : INT32_MAX); }

// The last of `sums` (ascending, n + 1 of them, the first 0) at or before x < sums[n].
__device__ __forceinline__ int32_t owner(const int32_t *sums, int32_t n, int32_t x) {
    int32_t b = 0, e = n;
    while (e - b > 1) {
        const int32_t m = (b + e) >> 1;
        if (sums[m] <= x) b = m;
        else e = m;
    }
    return b;
}

__global__ void __launch_bounds__(kThreads, 1) kv_plan_kernel(const __grid_constant__ KvPlanArgs a) {
    // [requests + 1] each: rows, pages begun and pages given back before a request's
    extern __shared__ int32_t sums_s[];
    __shared__ Sums warp_s[kWarps];
    __shared__ int32_t taken_s[kWarps];
    const int n = a.num_requests;
    int32_t *start = sums_s, *begun = start + n + 1, *back = begun + n + 1;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = static_cast<int>(cluster_rank()), threads = static_cast<int>(gridDim.x) * kThreads;
    const int tid = rank * kThreads + static_cast<int>(threadIdx.x);
    const bool first = rank == 0;
    pdl_wait();
    pdl_launch_dependents();
    const int32_t given = *a.free_count;
    const int32_t old = min(max(given, 0), a.free_capacity);
    if (old != given && tid == 0) report(a.status, DSA_ERR_BOUNDS);
    // ---- sums: every length is read once, side by side, then a thread takes neighbouring requests
    for (int i = threadIdx.x; i < n; i += kThreads) {
        const Request r = read_request(a, i);
        if (r.bad && first) report(a.status, DSA_ERR_BOUNDS);
        start[i] = static_cast<int32_t>(r.wide);
        begun[i] = r.need;
        back[i] = r.back;
    }
    __syncthreads();
    const int per = (n + kThreads - 1) / kThreads | 1;  // (odd: without bank conflicts)
    const int lo = min(n, static_cast<int>(threadIdx.x) * per), hi = min(n, lo + per);
    Sums mine = {0, 0, 0};
    for (int i = lo; i < hi; ++i) mine.add({begun[i], static_cast<uint32_t>(start[i]), back[i]});
    Sums upto = mine;
#pragma unroll 1
    for (int o = 1; o < 32; o <<= 1) {
        const Sums s = shifted(upto, o);
        if (lane >= o) upto.add(s);
    }
    if (lane == 31) warp_s[warp] = upto;
    __syncthreads();
    if (warp == 0) {
        Sums s = warp_s[lane];
#pragma unroll 1
        for (int o = 1; o < 32; o <<= 1) {
            const Sums u = shifted(s, o);
            if (lane >= o) s.add(u);
        }
        warp_s[lane] = s;
    }
    __syncthreads();
    const Sums total = warp_s[kWarps - 1];
    Sums at = {upto.need - mine.need, upto.wide - mine.wide, upto.back - mine.back};
    if (warp > 0) at.add(warp_s[warp - 1]);
    // what ended requests give back goes onto the stack first
    const int32_t count = static_cast<int32_t>(min(old + total.back, static_cast<int64_t>(a.free_capacity)));
    if (old + total.back > a.free_capacity && tid == 0) report(a.status, DSA_ERR_BOUNDS);
    const auto fits = [&](int32_t need, uint32_t wide, int64_t pages, int64_t rows) {  // with the sums behind the request
        return (need == 0 || pages <= count) && (wide == 0 || rows <= a.max_rows);
    };
    const auto granted = [&](const Request &r, int i) {
        return fits(r.need, r.wide, begun[i] + static_cast<int64_t>(r.need), start[i] + static_cast<int64_t>(r.wide));
    };
    bool denied = false;
    int32_t taken = 0;  // pages of those that get them: of all up to the first that does not
    for (int i = lo; i < hi; ++i) {
        const Sums r = {begun[i], static_cast<uint32_t>(start[i]), back[i]};
        start[i] = capped(at.wide);
        begun[i] = capped(at.need);
        back[i] = capped(at.back);
        at.add(r);
        const bool ok = fits(static_cast<int32_t>(r.need), static_cast<uint32_t>(r.wide), at.need, at.wide);
        denied |= !ok;
        if (ok && r.need > 0) taken = static_cast<int32_t>(at.need);
    }
    if (threadIdx.x == 0) {
        start[n] = capped(total.wide);
        begun[n] = capped(total.need);
        back[n] = capped(total.back);
    }
    if (denied && first && a.granted == nullptr) report(a.status, DSA_ERR_BOUNDS);
    taken = __reduce_max_sync(0xffffffffu, taken);
    if (lane == 0) taken_s[warp] = taken;
    __syncthreads();
    taken = __reduce_max_sync(0xffffffffu, taken_s[lane]);
    // ---- pages given back
    if (total.back > 0) {
        // a run of neighbours a warp, most of them of one request, and several on their way at once (one by one like the
        // rows: 103 us where half of 500 requests gave back 4,096 pages each, so 23)
        const int64_t all = count - old, per_warp = (all + threads - 1) / threads * 32, from = tid / 32 * per_warp;
        const int32_t end = static_cast<int32_t>(min(all, from + per_warp));
        for (int64_t t = from + lane; t < end;) {
            const int32_t i = owner(back, n, static_cast<int32_t>(t)), behind = min(end, back[i + 1]);
            const Request r = read_request(a, i);
            const int32_t *ids = a.block_table + i * a.bt_stride + (r.had - r.back - back[i]);
            for (; t < behind; t += 32 * kAtOnce) {
                int32_t id[kAtOnce];
#pragma unroll
                for (int k = 0; k < kAtOnce; ++k)
                    if (t + 32 * k < behind) id[k] = ids[t + 32 * k];
#pragma unroll
                for (int k = 0; k < kAtOnce; ++k)
                    if (t + 32 * k < behind) a.free_pages[old + t + 32 * k] = id[k];
            }
            t -= (t - behind) / 32 * 32;  // its first behind the request's
        }
        cluster_meet();
    }
    // ---- rows
    for (int row = tid; row < a.max_rows; row += threads) {
        int32_t req = 0, pos = -1, slot = -1;
        if (row < start[n]) {
            req = owner(start, n, row);
            const Request r = read_request(a, req);
            const int32_t j = row - start[req];
            if (j < r.fresh && granted(r, req)) {
                pos = r.ctx + j;
                const int32_t p = pos >> a.page_shift;
                const int32_t id = p < r.had ? a.block_table[req * a.bt_stride + p]
                                             : a.free_pages[count - 1 - (begun[req] + p - r.had)];
                if (id >= 0 && id < a.num_pages) slot = id * a.page_size + (pos & (a.page_size - 1));
                else report(a.status, DSA_ERR_BOUNDS);
            }
        }
        a.row_req[row] = req;
        a.row_ctx[row] = pos + 1;
        if (a.positions != nullptr) a.positions[row] = pos;
        if (a.slots != nullptr) a.slots[row] = slot;
    }
    // ---- table entries of the pages begun
    for (int t = tid; t < taken; t += threads) {
        const int32_t i = owner(begun, n, t);
        const Request r = read_request(a, i);
        a.block_table[i * a.bt_stride + r.had + (t - begun[i])] = a.free_pages[count - 1 - t];
    }
    cluster_meet();
    // ---- what may stand where it was read from (a thread reads the lengths that it alone replaces)
    for (int i = tid; i < n; i += threads) {
        const Request r = read_request(a, i);
        const int32_t fresh = granted(r, i) ? r.fresh : 0;
        if (a.granted != nullptr) a.granted[i] = fresh;
        if (a.context_out != nullptr) a.context_out[i] = r.ended ? 0 : r.ctx + fresh;
        if (a.row_start != nullptr) a.row_start[i] = min(start[i], a.max_rows);
    }
    for (int i = tid; i <= a.num_segments && a.num_segments > 0; i += threads) {
        int32_t req = a.segment_requests[i];
        if (req < 0 || req > n) {
            report(a.status, DSA_ERR_BOUNDS);
            req = req < 0 ? 0 : n;
        }
        a.segment_rows[i] = min(start[req], a.max_rows);
    }
    if (tid == 0) {
        if (a.row_start != nullptr) a.row_start[n] = min(start[n], a.max_rows);
        if (a.free_count_out != nullptr) *a.free_count_out = count - taken;
    }
}

}  // namespace

cudaError_t launch_kv_plan(const KvPlanArgs &a, cudaStream_t s) {
    const size_t smem = 3 * (static_cast<size_t>(a.num_requests) + 1) * 4;
    if (smem > 49152) {
        static std::atomic<uint64_t> configured{0};  // a bit a device
        int dev = 0;
        cudaError_t e = cudaGetDevice(&dev);
        if (e != cudaSuccess) return e;
        const uint64_t bit = 1ull << (dev & 63);
        if (dev >= 64 || !(configured.load() & bit)) {
            e = cudaFuncSetAttribute(kv_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     3 * (kPlanMaxRequests + 1) * 4);
            if (e != cudaSuccess) return e;
            if (dev < 64) configured.fetch_or(bit);
        }
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(kCtas);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = kCtas;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kv_plan_kernel, a);
}

}  // namespace dsa
