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
// keeps them in shared memory; a row finds its request there by bisection.  What one CTA writes and another reads (pages
// that ended requests give back) or what a call may update in place (contexts, the stack's count, which all CTAs read
// first) is set apart by cluster barriers.
#include "kernels.h"
#include "ptx.cuh"

namespace dsa {

namespace {

constexpr int kThreads = 1024, kWarps = kThreads / 32;

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

__device__ __forceinline__ int32_t capped(int64_t x, int32_t most) {
    return static_cast<int32_t>(x < most ? x : most);
}

__global__ void __launch_bounds__(kThreads, 1) kv_plan_kernel(const __grid_constant__ KvPlanArgs a) {
    // [requests + 1] first row of each; [requests] place among the pages begun (or -1: no tokens for it this time), or
    // among those given back
    extern __shared__ int32_t sums_s[];
    __shared__ Sums warp_s[kWarps];
    const int n = a.num_requests;
    int32_t *start = sums_s, *place = sums_s + n + 1;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = static_cast<int>(cluster_rank()), ctas = static_cast<int>(gridDim.x);
    const bool first = rank == 0;
    pdl_wait();
    pdl_launch_dependents();
    int32_t count = *a.free_count;
    if (count < 0 || count > a.free_capacity) {
        if (first && threadIdx.x == 0) report(a.status, DSA_ERR_BOUNDS);
        count = count < 0 ? 0 : a.free_capacity;
    }
    // ---- sums: a thread takes neighbouring requests
    const int per = (n + kThreads - 1) / kThreads, lo = min(n, static_cast<int>(threadIdx.x) * per), hi = min(n, lo + per);
    Sums mine = {0, 0, 0};
    for (int i = lo; i < hi; ++i) {
        const Request r = read_request(a, i);
        if (r.bad && first) report(a.status, DSA_ERR_BOUNDS);
        mine.add({r.need, r.wide, r.back});
    }
    Sums upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const Sums s = shifted(upto, o);
        if (lane >= o) upto.add(s);
    }
    if (lane == 31) warp_s[warp] = upto;
    __syncthreads();
    if (warp == 0) {
        Sums s = warp_s[lane];
#pragma unroll
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
    if (count + total.back > a.free_capacity && first && threadIdx.x == 0) report(a.status, DSA_ERR_BOUNDS);
    const int32_t old = count;
    count = capped(count + total.back, a.free_capacity);
    bool denied = false;
    for (int i = lo; i < hi; ++i) {
        const Request r = read_request(a, i);
        start[i] = capped(at.wide, a.max_rows);
        const bool fits = (r.need == 0 || at.need + r.need <= count) && (r.wide == 0 || at.wide + r.wide <= a.max_rows);
        denied |= !fits;
        place[i] = r.ended ? capped(at.back, INT32_MAX) : fits ? capped(at.need, INT32_MAX) : -1;
        at.add({r.need, r.wide, r.back});
    }
    if (threadIdx.x == 0) start[n] = capped(total.wide, a.max_rows);
    if (denied && first && a.granted == nullptr) report(a.status, DSA_ERR_BOUNDS);
    __syncthreads();
    // ---- pages given back: a warp a request
    const int warps = ctas * kWarps, my_warp = rank * kWarps + warp;
    if (total.back > 0) {
        for (int i0 = my_warp * 32; i0 < n; i0 += warps * 32) {
            const int i = i0 + lane;
            Request r = {};
            if (i < n) r = read_request(a, i);
            for (uint32_t some = __ballot_sync(0xffffffffu, r.back > 0); some != 0; some &= some - 1) {
                const int l = __ffs(some) - 1, j = i0 + l;
                const int32_t back = __shfl_sync(0xffffffffu, r.back, l), had = __shfl_sync(0xffffffffu, r.had, l);
                const int32_t *from = a.block_table + j * a.bt_stride + (had - back);
                for (int k = lane; k < back; k += 32) {
                    const int64_t to = static_cast<int64_t>(old) + place[j] + k;
                    if (to < a.free_capacity) a.free_pages[to] = from[k];
                }
            }
        }
        cluster_meet();
    }
    // ---- rows
    const auto page_of = [&](int i, const Request &r, int p) {
        return p < r.had ? a.block_table[i * a.bt_stride + p] : a.free_pages[count - 1 - (place[i] + p - r.had)];
    };
    const int threads = ctas * kThreads, tid = rank * kThreads + static_cast<int>(threadIdx.x);
    for (int row = tid; row < a.max_rows; row += threads) {
        int32_t req = 0, pos = -1, slot = -1;
        if (row < start[n]) {
            int b = 0, e = n;  // the last request that starts at or before the row
            while (e - b > 1) {
                const int m = (b + e) >> 1;
                if (start[m] <= row) b = m;
                else e = m;
            }
            req = b;
            const Request r = read_request(a, req);
            const int32_t j = row - start[req];
            if (j < r.fresh && place[req] >= 0) {
                pos = r.ctx + j;
                const int32_t id = page_of(req, r, pos >> a.page_shift);
                if (id >= 0 && id < a.num_pages) slot = id * a.page_size + (pos & (a.page_size - 1));
                else report(a.status, DSA_ERR_BOUNDS);
            }
        }
        a.row_req[row] = req;
        a.row_ctx[row] = pos + 1;
        if (a.positions != nullptr) a.positions[row] = pos;
        if (a.slots != nullptr) a.slots[row] = slot;
    }
    // ---- table entries of the pages begun: the first of each request by its lane, longer runs by the warp
    for (int i0 = my_warp * 32; i0 < n; i0 += warps * 32) {
        const int i = i0 + lane;
        Request r = {};
        if (i < n) r = read_request(a, i);
        const int32_t need = i < n && place[i] >= 0 ? r.need : 0;
        if (need > 0) a.block_table[i * a.bt_stride + r.had] = page_of(i, r, r.had);
        for (uint32_t some = __ballot_sync(0xffffffffu, need > 1); some != 0; some &= some - 1) {
            const int l = __ffs(some) - 1, j = i0 + l;
            const int32_t pages = __shfl_sync(0xffffffffu, need, l), had = __shfl_sync(0xffffffffu, r.had, l);
            for (int k = 1 + lane; k < pages; k += 32)
                a.block_table[j * a.bt_stride + had + k] = a.free_pages[count - 1 - (place[j] + k)];
        }
    }
    // ---- what may stand where it was read from
    int64_t taken = 0;  // the requests that get pages are those up to the first that does not
    for (int i = lo; i < hi; ++i) {
        const Request r = read_request(a, i);
        if (r.need > 0 && place[i] >= 0) taken = static_cast<int64_t>(place[i]) + r.need;
    }
    cluster_meet();
    for (int i = tid; i < n; i += threads) {
        // (a thread reads the lengths that it alone replaces)
        const Request r = read_request(a, i);
        const int32_t granted = place[i] >= 0 ? r.fresh : 0;
        if (a.granted != nullptr) a.granted[i] = granted;
        if (a.context_out != nullptr) a.context_out[i] = r.ended ? 0 : r.ctx + granted;
        if (a.row_start != nullptr) a.row_start[i] = start[i];
    }
    for (int i = tid; i <= a.num_segments && a.num_segments > 0; i += threads) {
        int32_t req = a.segment_requests[i];
        if (req < 0 || req > n) {
            report(a.status, DSA_ERR_BOUNDS);
            req = req < 0 ? 0 : n;
        }
        a.segment_rows[i] = start[req];
    }
    if (!first) return;
    if (threadIdx.x == 0 && a.row_start != nullptr) a.row_start[n] = start[n];
    // the largest `taken` of the threads
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) taken = max(taken, __shfl_xor_sync(0xffffffffu, taken, o));
    if (lane == 0) warp_s[warp].need = taken;
    __syncthreads();
    if (warp == 0) {
        taken = warp_s[lane].need;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) taken = max(taken, __shfl_xor_sync(0xffffffffu, taken, o));
        if (lane == 0 && a.free_count_out != nullptr) *a.free_count_out = count - static_cast<int32_t>(taken);
    }
}

}  // namespace

cudaError_t launch_kv_plan(const KvPlanArgs &a, cudaStream_t s) {
    const size_t smem = (2 * static_cast<size_t>(a.num_requests) + 1) * 4;
    cudaError_t e = cudaFuncSetAttribute(kv_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         static_cast<int>((2 * kPlanMaxRequests + 1) * 4));
    if (e != cudaSuccess) return e;
    // one CTA writes the few rows of a decode step sooner than eight that have to meet
    const unsigned ctas = a.max_rows > kPlanOneCtaRows || a.num_requests > kPlanOneCtaRows ? 8 : 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = ctas;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kv_plan_kernel, a);
}

}  // namespace dsa
