// kv_attention.cu -- dense attention of new tokens over the paged K/V pool (dsa_kv_attention).
//
//   out[r, h, :] = sum_t softmax_t(sm_scale <q[r,h,:], K_g,t>) V_g,t   over t < row_ctx[r]
//
// One CTA per (row, query head): each warp takes every fourth token, its lanes D / 32 dims each, with
// an online softmax in log2 units; the warps' (max, sum, output) are merged in shared memory.
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "kernels.h"
#include "ptx.cuh"

namespace dsa {

namespace {

constexpr int kWarps = 4;

__device__ __forceinline__ float kv_value(const uint8_t *pool, bool fp8, int64_t i) {
    if (fp8) {
        __nv_fp8_e4m3 v;
        v.__x = pool[i];
        return static_cast<float>(v);
    }
    return __bfloat162float(reinterpret_cast<const __nv_bfloat16 *>(pool)[i]);
}

template <int D>
__global__ void __launch_bounds__(kWarps * 32) kv_attention_kernel(const KvAttnArgs a) {
    constexpr int E = D / 32;
    __shared__ float sm_m[kWarps], sm_l[kWarps], sm_o[kWarps][D];
    pdl_wait();
    const int r = blockIdx.x / a.num_heads, h = blockIdx.x % a.num_heads;
    const int g = h / (a.num_heads / a.kv_heads);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int ctx = a.row_ctx[r];
    const int req = a.row_req[r];
    if (ctx < 0 || ctx > a.max_ctx || req < 0 || req >= a.num_requests || req != a.row_req[r - r % a.group]) {
        if (threadIdx.x == 0) report(a.status, DSA_ERR_BOUNDS);
        ctx = 0;
    }
    const uint16_t *q = a.q + r * a.q_stride + static_cast<int64_t>(h) * D + lane * E;
    float qv[E], o[E];
#pragma unroll
    for (int e = 0; e < E; ++e) {
        qv[e] = __uint_as_float(static_cast<uint32_t>(q[e]) << 16);
        o[e] = 0.f;
    }
    float m = -INFINITY, l = 0.f;
    for (int t = warp; t < ctx; t += kWarps) {
        const int32_t page = a.block_table[req * a.bt_stride + t / a.page_size];
        if (page < 0 || page >= a.num_pages) {
            if (lane == 0) report(a.status, DSA_ERR_BOUNDS);
            continue;
        }
        const int64_t k = ((static_cast<int64_t>(page) * a.kv_heads + g) * 2 * a.page_size + t % a.page_size) * D + lane * E;
        float s = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) s += qv[e] * kv_value(a.pool, a.fp8, k + e);
#pragma unroll
        for (int i = 16; i > 0; i >>= 1) s += __shfl_xor_sync(0xffffffffu, s, i);
        s *= a.s_scale;
        const float mn = fmaxf(m, s), base = mn == -INFINITY ? 0.f : mn;
        const float w = exp2f(m - base), p = exp2f(s - base);
        m = mn;
        l = l * w + p;
        const int64_t v = k + static_cast<int64_t>(a.page_size) * D;
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] = o[e] * w + p * kv_value(a.pool, a.fp8, v + e);
    }
    if (lane == 0) {
        sm_m[warp] = m;
        sm_l[warp] = l;
    }
#pragma unroll
    for (int e = 0; e < E; ++e) sm_o[warp][lane * E + e] = o[e];
    __syncthreads();
    if (threadIdx.x >= D) return;
    float M = -INFINITY;
    for (int w = 0; w < kWarps; ++w) M = fmaxf(M, sm_m[w]);
    const float base = M == -INFINITY ? 0.f : M;
    float sum = 0.f, x = 0.f;
    for (int w = 0; w < kWarps; ++w) {
        const float f = exp2f(sm_m[w] - base);
        sum += sm_l[w] * f;
        x += sm_o[w][threadIdx.x] * f;
    }
    const int64_t row = static_cast<int64_t>(r) * a.num_heads + h;
    const __nv_bfloat16 b = __float2bfloat16_rn(sum == 0.f ? 0.f : x / sum * a.v_scale);
    a.out[row * D + threadIdx.x] = __bfloat16_as_ushort(b);
    if (threadIdx.x == 0 && a.lse != nullptr) a.lse[row] = sum == 0.f ? -INFINITY : (base + log2f(sum)) * 0.6931471805599453f;
}

}  // namespace

cudaError_t launch_kv_attention(const KvAttnArgs &a, cudaStream_t s) {
    if (a.num_rows == 0) return cudaSuccess;
    const int64_t grid = static_cast<int64_t>(a.num_rows) * a.num_heads;
    if (grid > 0x7fffffff) return cudaErrorInvalidConfiguration;
    const dim3 g(static_cast<unsigned>(grid)), b(kWarps * 32);
    return a.head_dim == 64 ? launch_pdl(kv_attention_kernel<64>, g, b, 0, s, a)
                            : launch_pdl(kv_attention_kernel<128>, g, b, 0, s, a);
}

size_t kv_attention_workspace_bytes(int64_t, int32_t, int32_t, int32_t, int32_t) { return 0; }

}  // namespace dsa
