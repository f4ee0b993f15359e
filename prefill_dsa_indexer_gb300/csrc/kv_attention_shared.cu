// kv_attention_shared.cu -- attention of a batch whose rows share prefixes (dsa_kv_attention_shared).
//
// This form lets every row read all of its tokens by itself (kv_attention.cu): right for every case, and as slow as
// if nothing were shared.  The segments are checked only.
#include "kv_attention_common.cuh"

namespace dsa {

namespace {

constexpr int kThreads = 1024;

__global__ void __launch_bounds__(kThreads, 1) kv_segments_kernel(const __grid_constant__ KvSegmentArgs a) {
    pdl_wait();
    pdl_launch_dependents();
    // a segment begins at or behind every bound before it
    __shared__ int32_t tops[kThreads];
    const int per = (a.num_segments + kThreads) / kThreads, lo = min(a.num_segments + 1, static_cast<int>(threadIdx.x) * per);
    const int hi = min(a.num_segments + 1, lo + per);
    int32_t top = INT32_MIN;
    for (int i = lo; i < hi; ++i) top = max(top, a.first_row[i]);
    tops[threadIdx.x] = top;
    __syncthreads();
    top = INT32_MIN;
    for (int t = 0; t < static_cast<int>(threadIdx.x) && lo < hi; ++t) top = max(top, tops[t]);
    for (int s = lo; s < min(hi, a.num_segments); ++s) {
        const int32_t first = a.first_row[s], end = a.first_row[s + 1];
        if (first < 0 || first < top || end < first || end > a.num_rows || first % a.group != 0 || end % a.group != 0 ||
            a.shared_ctx[s] < 0)
            report(a.status, DSA_ERR_BOUNDS);
        top = max(top, first);
    }
}

}  // namespace

cudaError_t launch_kv_attention_shared(const KvSegmentArgs &seg, KvAttnArgs &a, void *workspace, cudaStream_t s) {
    if (a.num_rows == 0) return cudaSuccess;
    const cudaError_t e = launch_pdl(kv_segments_kernel, dim3(1), dim3(kThreads), 0, s, seg);
    return e != cudaSuccess ? e : launch_kv_attention(a, workspace, s);
}

}  // namespace dsa
