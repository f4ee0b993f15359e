// kv_shares.cu -- kv_share by itself (tests/test_gpu_kv_shares.py): which CTA takes which share of the rows' own tokens.
#include "kv_attention_common.cuh"

// A CTA with a share stays for `linger` cycles, as one that works; made[share] counts who took it, by[cta] is its share.
__global__ void shares_kernel(int32_t *own_sms, int32_t *made, int32_t *by, int32_t linger) {
    __shared__ dsa::kv::KvSchedule sched;
    if (threadIdx.x < 32) dsa::kv::kv_share(own_sms, &sched, threadIdx.x);
    __syncthreads();
    if (threadIdx.x > 0) return;
    by[blockIdx.x] = sched.mine;
    if (sched.mine < 0 || sched.mine >= static_cast<int>(gridDim.x)) return;
    atomicAdd(made + sched.mine, 1);
    const long long t0 = clock64();
    while (clock64() - t0 < linger) {
    }
}

extern "C" int shares_launch(void *own_sms, void *made, void *by, int32_t linger, int32_t ctas, int32_t smem, void *stream) {
    cudaError_t e = cudaFuncSetAttribute(shares_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    shares_kernel<<<ctas, 128, smem, static_cast<cudaStream_t>(stream)>>>(
        static_cast<int32_t *>(own_sms), static_cast<int32_t *>(made), static_cast<int32_t *>(by), linger);
    return cudaGetLastError();
}
