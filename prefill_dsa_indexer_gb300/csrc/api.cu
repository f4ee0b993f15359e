// api.cu -- the extern "C" entry points of libdsa declared in include/dsa.h.
//
// Each call validates its arguments on the host, encodes the TMA tensor maps
// it needs, and enqueues its kernels on the caller's stream.  Nothing here
// allocates device memory or synchronises with the device.
#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <cmath>
#include <cstdint>
#include <cstring>
#include <mutex>

#include "../../include/dsa.h"
#include "kernels.h"
#include "ptx.cuh"

namespace dsa {

namespace {

static_assert(DSA_HIST_BINS == kHistBins, "the header and the kernels agree on the histogram size");

PFN_cuTensorMapEncodeTiled_v12000 get_encoder() {
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    });
    return fn;
}

// 2D byte tensor [rows, 128 B] with a [box_rows, 128 B] box, 128-byte swizzle.
bool encode_rows128(CUtensorMap *map, const void *base, uint64_t rows, uint32_t box_rows) {
    auto enc = get_encoder();
    if (enc == nullptr) return false;
    const cuuint64_t dims[2] = {128, rows};
    const cuuint64_t strides[1] = {128};
    const cuuint32_t box[2] = {128, box_rows};
    const cuuint32_t estr[2] = {1, 1};
    CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void *>(base), dims, strides, box, estr,
                     CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS;
}

// 2D tensor of 4-bit values [rows, 128] with 64-byte rows (MXFP4 index keys), a [box_rows, 128]
// box landing in shared memory as 128-byte rows (each 16 values in the low 8 bytes of a 16-byte
// unit, the layout 4-bit tensor-core operands take), 128-byte swizzle.  Base: 32-byte aligned.
bool encode_fp4_rows64(CUtensorMap *map, const void *base, uint64_t rows, uint32_t box_rows) {
    auto enc = get_encoder();
    if (enc == nullptr) return false;
    const cuuint64_t dims[2] = {128, rows};
    const cuuint64_t strides[1] = {64};
    const cuuint32_t box[2] = {128, box_rows};
    const cuuint32_t estr[2] = {1, 1};
    CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_16U4_ALIGN16B, 2, const_cast<void *>(base), dims, strides, box,
                     estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                     CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS;
}

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

int check_rows(const dsa_rows *rows) {
    if (rows == nullptr) return DSA_ERR_INVALID_ARG;
    if (rows->num_rows < 0 || rows->max_ctx < 0 || rows->num_requests < 0) return DSA_ERR_INVALID_ARG;
    if (rows->num_rows == 0) return DSA_OK;
    if (!rows->block_table || !rows->row_req || !rows->row_ctx) return DSA_ERR_INVALID_ARG;
    const int64_t need_pages = (static_cast<int64_t>(rows->max_ctx) + DSA_PAGE_SIZE - 1) / DSA_PAGE_SIZE;
    if (rows->bt_stride < need_pages) return DSA_ERR_INVALID_ARG;
    return DSA_OK;
}

int launch_status(cudaError_t e) { return e == cudaSuccess ? DSA_OK : DSA_ERR_CUDA; }

}  // namespace

bool encode_rows128_map(CUtensorMap *map, const void *base, uint64_t rows, uint32_t box_rows) {
    return encode_rows128(map, base, rows, box_rows);
}

// 2D byte tensor [rows, row_bytes] of a K/V pool (64, 128 or 256 bytes a row) with a box of box_rows rows by
// one swizzle span (64 or 128 bytes).
bool encode_kv_rows_map(CUtensorMap *map, const void *base, uint64_t rows, uint32_t row_bytes, uint32_t box_rows) {
    auto enc = get_encoder();
    if (enc == nullptr) return false;
    const cuuint64_t dims[2] = {row_bytes, rows};
    const cuuint64_t strides[1] = {row_bytes};
    const cuuint32_t box[2] = {row_bytes < 128 ? row_bytes : 128, box_rows};
    const cuuint32_t estr[2] = {1, 1};
    CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void *>(base), dims, strides, box, estr,
                     CU_TENSOR_MAP_INTERLEAVE_NONE,
                     row_bytes < 128 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
                     CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS;
}

int device_sm_count() {
    static int counts[64] = {0};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 0;
    if (dev < 0 || dev >= 64) return 0;
    if (counts[dev] == 0) {
        int n = 0;
        cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
        counts[dev] = n;
    }
    return counts[dev];
}

}  // namespace dsa

using namespace dsa;

extern "C" {

int dsa_version(void) { return 100; }

const char *dsa_status_string(int status) {
    switch (status) {
        case DSA_OK: return "ok";
        case DSA_ERR_INVALID_ARG: return "invalid argument";
        case DSA_ERR_UNSUPPORTED: return "unsupported configuration";
        case DSA_ERR_CUDA: return "CUDA error";
        case DSA_ERR_WORKSPACE: return "workspace too small";
        case DSA_ERR_TIMEOUT: return "device wait timed out";
        case DSA_ERR_BOUNDS: return "index out of bounds in device data";
        case DSA_ERR_RANGE: return "value out of representable range";
        default: return "unknown status";
    }
}

static int indexer_common(const dsa_cache *index_cache, const dsa_rows *rows, const uint8_t *q_idx,
                          const float *head_w, float *logits, int64_t logits_stride, uint32_t *hist,
                          int32_t *dev_status, void *stream) {
    if (index_cache == nullptr) return DSA_ERR_INVALID_ARG;
    int rc = check_rows(rows);
    if (rc != DSA_OK) return rc;
    if (index_cache->page_size != DSA_PAGE_SIZE) return DSA_ERR_UNSUPPORTED;
    if (index_cache->format != DSA_KEY_FP8 && index_cache->format != DSA_KEY_MXFP4) return DSA_ERR_UNSUPPORTED;
    const bool mx = index_cache->format == DSA_KEY_MXFP4;
    const int G = rows->rows_per_group;
    if (G != 1 && G != 2 && G != 4 && G != 8) return DSA_ERR_UNSUPPORTED;
    if (rows->num_rows % G != 0) return DSA_ERR_INVALID_ARG;
    if (rows->num_rows == 0) return DSA_OK;
    if (!index_cache->base || index_cache->num_pages <= 0 || !q_idx || !head_w || !logits)
        return DSA_ERR_INVALID_ARG;
    if (!aligned(index_cache->base, mx ? 32 : 16) || !aligned(q_idx, 16)) return DSA_ERR_INVALID_ARG;
    if (logits_stride < rows->max_ctx) return DSA_ERR_INVALID_ARG;
    const uint64_t pool_rows = static_cast<uint64_t>(index_cache->num_pages) * (mx ? 68u : 66u);
    if (pool_rows >= (1ull << 31)) return DSA_ERR_UNSUPPORTED;
    const int sms = device_sm_count();
    if (sms <= 0) return DSA_ERR_CUDA;

    CUtensorMap key_map, q_map;
    if (mx ? !encode_fp4_rows64(&key_map, index_cache->base, pool_rows, DSA_PAGE_SIZE)
           : !encode_rows128(&key_map, index_cache->base, pool_rows, DSA_PAGE_SIZE))
        return DSA_ERR_CUDA;
    if (!encode_rows128(&q_map, q_idx, static_cast<uint64_t>(rows->num_rows) * DSA_INDEX_HEADS,
                        static_cast<uint32_t>(G * DSA_INDEX_HEADS)))
        return DSA_ERR_CUDA;
    IndexerArgs a;
    a.pool = static_cast<const uint8_t *>(index_cache->base);
    a.num_pages = index_cache->num_pages;
    a.block_table = rows->block_table;
    a.bt_stride = rows->bt_stride;
    a.num_requests = rows->num_requests;
    a.row_req = rows->row_req;
    a.row_ctx = rows->row_ctx;
    a.max_ctx = rows->max_ctx;
    a.head_w = head_w;
    a.logits = logits;
    a.logits_stride = logits_stride;
    a.status = dev_status;
    a.hist = hist;
    const int num_groups = rows->num_rows / G;
    for (int g0 = 0; g0 < num_groups; g0 += kIndexerMaxGroups) {
        a.group0 = g0;
        a.num_groups = num_groups - g0 < kIndexerMaxGroups ? num_groups - g0 : kIndexerMaxGroups;
        cudaError_t e = launch_indexer(key_map, q_map, a, mx, G, sms, static_cast<cudaStream_t>(stream));
        if (e != cudaSuccess) return DSA_ERR_CUDA;
    }
    return DSA_OK;
}

int dsa_indexer_logits(const dsa_cache *index_cache, const dsa_rows *rows, const uint8_t *q_idx,
                       const float *head_w, float *logits, int64_t logits_stride, int32_t *dev_status,
                       void *stream) {
    return indexer_common(index_cache, rows, q_idx, head_w, logits, logits_stride, nullptr, dev_status, stream);
}

int dsa_indexer_logits_hist(const dsa_cache *index_cache, const dsa_rows *rows, const uint8_t *q_idx,
                            const float *head_w, float *logits, int64_t logits_stride, uint32_t *hist,
                            int32_t *dev_status, void *stream) {
    if (hist == nullptr && rows != nullptr && rows->num_rows > 0) return DSA_ERR_INVALID_ARG;
    return indexer_common(index_cache, rows, q_idx, head_w, logits, logits_stride, hist, dev_status, stream);
}

static int topk_common(const float *logits, int64_t logits_stride, const int32_t *row_ctx, int32_t num_rows,
                       int32_t max_ctx, int32_t k, uint32_t *hist, bool discard, int32_t *idx_out,
                       int32_t *dev_status, void *stream, const dsa_rows *slot_rows = nullptr,
                       int64_t pool_pages = 0, int32_t *slots_out = nullptr, const uint8_t *warm_pool = nullptr,
                       void *workspace = nullptr, size_t workspace_bytes = 0) {
    if (num_rows < 0 || max_ctx < 0) return DSA_ERR_INVALID_ARG;
    if (k < 1 || k > DSA_MAX_TOPK) return DSA_ERR_UNSUPPORTED;
    if (num_rows == 0) return DSA_OK;
    if (!logits || !row_ctx || !idx_out || logits_stride < max_ctx) return DSA_ERR_INVALID_ARG;
    TopkArgs a{logits, logits_stride, row_ctx, num_rows, max_ctx, k, idx_out, dev_status, hist, discard,
               nullptr, nullptr, 0, nullptr, 0, 0};
    if (workspace != nullptr && hist == nullptr) {
        // with a large enough workspace, few long rows take the histogram selection
        const TopkChunkPlan p = topk_chunk_plan(num_rows, max_ctx, k, device_sm_count());
        if (p.bytes > 0) {
            if (workspace_bytes < p.bytes) return DSA_ERR_WORKSPACE;
            if (!aligned(workspace, 256)) return DSA_ERR_INVALID_ARG;
            topk_chunk_bind(a, p, workspace);
        }
    }
    if (slots_out != nullptr) {
        if (slot_rows == nullptr || pool_pages <= 0) return DSA_ERR_INVALID_ARG;
        if (pool_pages * DSA_PAGE_SIZE > INT32_MAX) return DSA_ERR_UNSUPPORTED;
        a.slots_out = slots_out;
        a.block_table = slot_rows->block_table;
        a.bt_stride = slot_rows->bt_stride;
        a.row_req = slot_rows->row_req;
        a.num_requests = slot_rows->num_requests;
        a.pool_pages = pool_pages;
        a.warm_pool = warm_pool;
    }
    return launch_status(launch_topk(a, static_cast<cudaStream_t>(stream)));
}

size_t dsa_topk_workspace_size(int32_t num_rows, int32_t max_ctx, int32_t k) {
    return topk_chunk_plan(num_rows, max_ctx, k, device_sm_count()).bytes;
}

int dsa_topk_slots_warm(const float *logits, int64_t logits_stride, const dsa_rows *rows, const dsa_cache *latent_cache,
                        int32_t k, int32_t *idx_out, int32_t *slots_out, int32_t *dev_status, void *workspace,
                        size_t workspace_bytes, void *stream) {
    int rc = check_rows(rows);
    if (rc != DSA_OK) return rc;
    if (latent_cache == nullptr || latent_cache->page_size != DSA_PAGE_SIZE) return DSA_ERR_INVALID_ARG;
    if (rows->num_rows > 0 && (slots_out == nullptr || latent_cache->base == nullptr)) return DSA_ERR_INVALID_ARG;
    if (!aligned(latent_cache->base, 16)) return DSA_ERR_INVALID_ARG;
    // FP8 rows are one contiguous 576-byte run each; NVFP4 tokens are spread over a page, not warmed
    const uint8_t *warm =
        latent_cache->format == DSA_LATENT_FP8 ? static_cast<const uint8_t *>(latent_cache->base) : nullptr;
    if (latent_cache->format != DSA_LATENT_FP8 && latent_cache->format != DSA_LATENT_NVFP4) return DSA_ERR_UNSUPPORTED;
    return topk_common(logits, logits_stride, rows->row_ctx, rows->num_rows, rows->max_ctx, k, nullptr, false,
                       idx_out, dev_status, stream, rows, latent_cache->num_pages, slots_out, warm, workspace,
                       workspace_bytes);
}

int dsa_topk_slots(const float *logits, int64_t logits_stride, const dsa_rows *rows, int64_t pool_pages, int32_t k,
                   int32_t *idx_out, int32_t *slots_out, int32_t *dev_status, void *workspace, size_t workspace_bytes,
                   void *stream) {
    int rc = check_rows(rows);
    if (rc != DSA_OK) return rc;
    if (rows->num_rows > 0 && slots_out == nullptr) return DSA_ERR_INVALID_ARG;
    return topk_common(logits, logits_stride, rows->row_ctx, rows->num_rows, rows->max_ctx, k, nullptr, false,
                       idx_out, dev_status, stream, rows, pool_pages, slots_out, nullptr, workspace, workspace_bytes);
}

int dsa_topk(const float *logits, int64_t logits_stride, const int32_t *row_ctx, int32_t num_rows,
             int32_t max_ctx, int32_t k, int32_t *idx_out, int32_t *dev_status, void *workspace,
             size_t workspace_bytes, void *stream) {
    return topk_common(logits, logits_stride, row_ctx, num_rows, max_ctx, k, nullptr, false, idx_out, dev_status,
                       stream, nullptr, 0, nullptr, nullptr, workspace, workspace_bytes);
}

int dsa_topk_hist(const float *logits, int64_t logits_stride, const int32_t *row_ctx, int32_t num_rows,
                  int32_t max_ctx, int32_t k, uint32_t *hist, int32_t *idx_out, int32_t *dev_status, void *stream) {
    if (hist == nullptr && num_rows > 0) return DSA_ERR_INVALID_ARG;
    return topk_common(logits, logits_stride, row_ctx, num_rows, max_ctx, k, hist, false, idx_out, dev_status,
                       stream);
}

// Workspace of dsa_indexer_topk: [histogram rows x DSA_HIST_BINS u32][logits rows x stride fp32],
// the logits row stride rounded up to 32 floats (128-byte rows).
static int64_t fused_logits_stride(int32_t max_ctx) { return (static_cast<int64_t>(max_ctx) + 31) / 32 * 32; }

size_t dsa_indexer_topk_workspace_size(int32_t num_rows, int32_t max_ctx) {
    if (num_rows <= 0 || max_ctx <= 0) return 0;
    return align256(static_cast<size_t>(num_rows) * DSA_HIST_BINS * 4) +
           align256(static_cast<size_t>(num_rows) * static_cast<size_t>(fused_logits_stride(max_ctx)) * 4);
}

int dsa_indexer_topk(const dsa_cache *index_cache, const dsa_rows *rows, const uint8_t *q_idx, const float *head_w,
                     int32_t k, int32_t *idx_out, int32_t *dev_status, void *workspace, size_t workspace_bytes,
                     void *stream) {
    int rc = check_rows(rows);
    if (rc != DSA_OK) return rc;
    if (k < 1 || k > DSA_MAX_TOPK) return DSA_ERR_UNSUPPORTED;
    if (rows->num_rows == 0) return DSA_OK;
    if (workspace == nullptr || !aligned(workspace, 256) ||
        workspace_bytes < dsa_indexer_topk_workspace_size(rows->num_rows, rows->max_ctx))
        return DSA_ERR_WORKSPACE;
    uint32_t *hist = static_cast<uint32_t *>(workspace);
    float *logits = reinterpret_cast<float *>(static_cast<uint8_t *>(workspace) +
                                              align256(static_cast<size_t>(rows->num_rows) * DSA_HIST_BINS * 4));
    const int64_t stride = fused_logits_stride(rows->max_ctx);
    rc = indexer_common(index_cache, rows, q_idx, head_w, logits, stride, hist, dev_status, stream);
    if (rc != DSA_OK) return rc;
    return topk_common(logits, stride, rows->row_ctx, rows->num_rows, rows->max_ctx, k, hist, true, idx_out,
                       dev_status, stream);
}

int dsa_page_to_slot(const dsa_rows *rows, int64_t pool_pages, const int32_t *idx, int32_t k, int32_t *slots,
                     int32_t *dev_status, void *stream) {
    int rc = check_rows(rows);
    if (rc != DSA_OK) return rc;
    if (k < 1) return DSA_ERR_INVALID_ARG;
    if (rows->num_rows == 0) return DSA_OK;
    if (!idx || !slots || pool_pages <= 0) return DSA_ERR_INVALID_ARG;
    if (pool_pages * DSA_PAGE_SIZE > INT32_MAX) return DSA_ERR_UNSUPPORTED;
    SlotArgs a{rows->block_table, rows->bt_stride, rows->num_requests, rows->row_req, rows->row_ctx, rows->num_rows,
               rows->max_ctx, pool_pages, idx, k, slots, dev_status};
    return launch_status(launch_page_to_slot(a, static_cast<cudaStream_t>(stream)));
}

size_t dsa_sparse_mla_workspace_size(int32_t num_rows, int32_t num_heads, int32_t k) {
    if (num_rows <= 0 || num_heads <= 0 || k <= 0) return 0;
    return mla_workspace_bytes(num_rows, num_heads, k);
}


enum class MlaMode { kPrefill, kDecode, kDecodePrepareOnly, kDecodePrepared };

static int sparse_mla_common(const dsa_cache *lat, const uint16_t *q, int32_t num_heads, const int32_t *slots,
                             int32_t num_rows, int32_t k, float sm_scale, float *out, float *lse,
                             int32_t *dev_status, void *ws, size_t ws_bytes, void *stream, MlaMode mode) {
    const bool decode = mode != MlaMode::kPrefill;
    const bool prep_only = mode == MlaMode::kDecodePrepareOnly;
    if (lat == nullptr || num_rows < 0) return DSA_ERR_INVALID_ARG;
    if (lat->page_size != DSA_PAGE_SIZE) return DSA_ERR_UNSUPPORTED;
    if (lat->format != DSA_LATENT_FP8 && lat->format != DSA_LATENT_NVFP4) return DSA_ERR_UNSUPPORTED;
    if (num_heads < 16 || num_heads > 96 || num_heads % 16 != 0) return DSA_ERR_UNSUPPORTED;
    if (k < 1) return DSA_ERR_INVALID_ARG;
    if (num_rows == 0) return DSA_OK;
    if (!lat->base || lat->num_pages <= 0 || !q || (!prep_only && (!slots || !out))) return DSA_ERR_INVALID_ARG;
    if (!aligned(lat->base, 16) || !aligned(q, 16)) return DSA_ERR_INVALID_ARG;
    if (!std::isfinite(sm_scale) || !std::isfinite(lat->tensor_scale)) return DSA_ERR_INVALID_ARG;
    MlaArgs a{};
    a.pool = static_cast<const uint8_t *>(lat->base);
    a.format = lat->format;
    a.num_pages = lat->num_pages;
    a.tensor_scale = lat->tensor_scale;
    a.q = q;
    a.num_heads = num_heads;
    a.slots = slots;
    a.num_rows = num_rows;
    a.k = k;
    a.sm_scale = sm_scale;
    a.out = out;
    a.lse = lse;
    a.status = dev_status;
    a.splits = 1;
    if (decode) {
        const size_t splits = mla_splits(static_cast<size_t>(k));
        if (splits > static_cast<size_t>(kMlaMaxSplits)) return DSA_ERR_UNSUPPORTED;
        if (splits > 1) {
            const size_t need = mla_workspace_bytes(num_rows, num_heads, k);
            if (ws == nullptr || ws_bytes < need) return DSA_ERR_WORKSPACE;
            if (!aligned(ws, 256)) return DSA_ERR_INVALID_ARG;
            uint8_t *w = static_cast<uint8_t *>(ws);
            a.part_o = reinterpret_cast<uint16_t *>(w);
            w += mla_part_o_bytes(num_rows, num_heads, splits);
            a.part_ml = reinterpret_cast<float *>(w);
            w += mla_part_ml_bytes(num_rows, num_heads, splits);
            a.qprep = w;
            a.splits = static_cast<int32_t>(splits);
        }
    }
    // split decode over FP8 latents runs on the FP8 tensor cores (mla_fp8.cu); NVFP4 latents,
    // prefill and single-part decode decode the latents to fp16 (mla.cu)
    const bool fp8_decode = decode && a.splits > 1 && lat->format == DSA_LATENT_FP8;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (prep_only) return launch_status(fp8_decode ? launch_mla_qprep_fp8(a, st) : launch_mla_qprep(a, st));
    a.q_prepared = mode == MlaMode::kDecodePrepared;
    return launch_status(fp8_decode ? launch_sparse_mla_fp8_decode(a, st) : launch_sparse_mla(a, st));
}

int dsa_sparse_mla_decode(const dsa_cache *latent_cache, const uint16_t *q, int32_t num_heads,
                          const int32_t *slots, int32_t num_rows, int32_t k, float sm_scale, float *out,
                          float *lse, int32_t *dev_status, void *workspace, size_t workspace_bytes, void *stream) {
    return sparse_mla_common(latent_cache, q, num_heads, slots, num_rows, k, sm_scale, out, lse, dev_status,
                             workspace, workspace_bytes, stream, MlaMode::kDecode);
}

int dsa_sparse_mla_decode_prepare(const dsa_cache *latent_cache, const uint16_t *q, int32_t num_heads,
                                  int32_t num_rows, int32_t k, int32_t *dev_status, void *workspace,
                                  size_t workspace_bytes, void *stream) {
    return sparse_mla_common(latent_cache, q, num_heads, nullptr, num_rows, k, 1.0f, nullptr, nullptr, dev_status,
                             workspace, workspace_bytes, stream, MlaMode::kDecodePrepareOnly);
}

int dsa_sparse_mla_decode_prepared(const dsa_cache *latent_cache, const uint16_t *q, int32_t num_heads,
                                   const int32_t *slots, int32_t num_rows, int32_t k, float sm_scale, float *out,
                                   float *lse, int32_t *dev_status, void *workspace, size_t workspace_bytes,
                                   void *stream) {
    return sparse_mla_common(latent_cache, q, num_heads, slots, num_rows, k, sm_scale, out, lse, dev_status,
                             workspace, workspace_bytes, stream, MlaMode::kDecodePrepared);
}

int dsa_sparse_mla_prefill(const dsa_cache *latent_cache, const uint16_t *q, int32_t num_heads,
                           const int32_t *slots, int32_t num_rows, int32_t k, float sm_scale, float *out,
                           float *lse, int32_t *dev_status, void *workspace, size_t workspace_bytes,
                           void *stream) {
    return sparse_mla_common(latent_cache, q, num_heads, slots, num_rows, k, sm_scale, out, lse, dev_status,
                             workspace, workspace_bytes, stream, MlaMode::kPrefill);
}

int dsa_cache_insert(const dsa_cache *index_cache, const dsa_cache *latent_cache, const int32_t *slots,
                     int32_t num_tokens, const uint16_t *index_keys, const uint16_t *latents, int32_t *dev_status,
                     void *stream) {
    if (index_cache == nullptr || latent_cache == nullptr || num_tokens < 0) return DSA_ERR_INVALID_ARG;
    if (index_cache->page_size != DSA_PAGE_SIZE || latent_cache->page_size != DSA_PAGE_SIZE) return DSA_ERR_UNSUPPORTED;
    if (index_cache->format != DSA_KEY_FP8 && index_cache->format != DSA_KEY_MXFP4) return DSA_ERR_UNSUPPORTED;
    if (latent_cache->format != DSA_LATENT_FP8 && latent_cache->format != DSA_LATENT_NVFP4) return DSA_ERR_UNSUPPORTED;
    if (num_tokens == 0) return DSA_OK;
    if (!index_cache->base || !latent_cache->base || !slots || !index_keys || !latents) return DSA_ERR_INVALID_ARG;
    if (index_cache->num_pages != latent_cache->num_pages || index_cache->num_pages <= 0) return DSA_ERR_INVALID_ARG;
    if (!aligned(index_cache->base, 16) || !aligned(latent_cache->base, 16) || !aligned(index_keys, 16) ||
        !aligned(latents, 16))
        return DSA_ERR_INVALID_ARG;
    if (!std::isfinite(latent_cache->tensor_scale) || !(latent_cache->tensor_scale > 0.f)) return DSA_ERR_INVALID_ARG;
    InsertArgs a;
    a.idx_pool = static_cast<uint8_t *>(const_cast<void *>(index_cache->base));
    a.key_fmt = index_cache->format;
    a.lat_pool = static_cast<uint8_t *>(const_cast<void *>(latent_cache->base));
    a.lat_fmt = latent_cache->format;
    a.tensor_scale = latent_cache->tensor_scale;
    a.num_pages = index_cache->num_pages;
    a.slots = slots;
    a.num_tokens = num_tokens;
    a.keys = index_keys;
    a.latents = latents;
    a.status = dev_status;
    return launch_status(launch_cache_insert(a, static_cast<cudaStream_t>(stream)));
}

// ------------------------------------------------------------------ failure-path self-test

static __global__ void wait_timeout_kernel(int32_t *status) {
    __shared__ uint64_t bar;
    __shared__ int abort_flag;
    if (threadIdx.x == 0) {
        abort_flag = 0;
        mbar_init(&bar, 1);  // one arrival that never comes
        fence_mbar_init();
    }
    __syncthreads();
    // lane 0 of every warp waits: the first to reach the limit reports and raises the abort
    // flag, the others then return at once
    if ((threadIdx.x & 31) == 0) mbar_wait(&bar, 0, &abort_flag, status);
    __syncthreads();
}

int dsa_selftest_wait_timeout(int32_t *dev_status, void *stream) {
    if (dev_status == nullptr) return DSA_ERR_INVALID_ARG;
    wait_timeout_kernel<<<1, 128, 0, static_cast<cudaStream_t>(stream)>>>(dev_status);
    return launch_status(cudaGetLastError());
}

// ------------------------------------------------------------------ MSA block-sparse variant

static int msa_check_rows(const dsa_rows *rows) {
    if (rows == nullptr) return DSA_ERR_INVALID_ARG;
    if (rows->num_rows < 0 || rows->max_ctx < 0 || rows->num_requests < 0) return DSA_ERR_INVALID_ARG;
    if (rows->num_rows == 0) return DSA_OK;
    if (!rows->block_table || !rows->row_req || !rows->row_ctx) return DSA_ERR_INVALID_ARG;
    const int64_t need_pages = (static_cast<int64_t>(rows->max_ctx) + DSA_MSA_PAGE - 1) / DSA_MSA_PAGE;
    if (rows->bt_stride < need_pages) return DSA_ERR_INVALID_ARG;
    return DSA_OK;
}

int dsa_msa_block_scores(const void *index_pool, int64_t num_pages, const dsa_rows *rows, const uint8_t *q_idx,
                         float *scores, int64_t score_stride, int32_t *dev_status, void *stream) {
    int rc = msa_check_rows(rows);
    if (rc != DSA_OK || rows->num_rows == 0) return rc;
    const int G = rows->rows_per_group;
    if (G != 1 && G != 2 && G != 4 && G != 8) return DSA_ERR_UNSUPPORTED;
    if (rows->num_rows % G != 0) return DSA_ERR_INVALID_ARG;
    if (!index_pool || num_pages <= 0 || !q_idx || !scores) return DSA_ERR_INVALID_ARG;
    if (!aligned(index_pool, 16) || !aligned(q_idx, 16)) return DSA_ERR_INVALID_ARG;
    const int64_t max_blocks = (static_cast<int64_t>(rows->max_ctx) + DSA_MSA_PAGE - 1) / DSA_MSA_PAGE;
    if (score_stride < max_blocks) return DSA_ERR_INVALID_ARG;
    const uint64_t pool_rows = static_cast<uint64_t>(num_pages) * DSA_MSA_PAGE;
    if (pool_rows >= (1ull << 31)) return DSA_ERR_UNSUPPORTED;
    const int sms = device_sm_count();
    if (sms <= 0) return DSA_ERR_CUDA;
    CUtensorMap key_map, q_map;
    const uint32_t q_box = static_cast<uint32_t>(G * DSA_MSA_GROUPS < 16 ? 16 : G * DSA_MSA_GROUPS);
    if (!encode_rows128(&key_map, index_pool, pool_rows, DSA_MSA_PAGE)) return DSA_ERR_CUDA;
    if (!encode_rows128(&q_map, q_idx, static_cast<uint64_t>(rows->num_rows) * DSA_MSA_GROUPS, q_box))
        return DSA_ERR_CUDA;
    const int num_groups = rows->num_rows / G;
    // pages per CTA: two CTAs per SM cover the rows' pages in about one wave (4..64 pages each)
    const int64_t total_pages = static_cast<int64_t>(num_groups) * (max_blocks > 0 ? max_blocks : 1);
    int64_t cp = (total_pages + 2 * sms - 1) / (2 * sms);
    cp = cp < 4 ? 4 : (cp > 64 ? 64 : cp);
    MsaScoreArgs a;
    a.num_pages = num_pages;
    a.block_table = rows->block_table;
    a.bt_stride = rows->bt_stride;
    a.num_requests = rows->num_requests;
    a.row_req = rows->row_req;
    a.row_ctx = rows->row_ctx;
    a.max_ctx = rows->max_ctx;
    a.chunk_pages = static_cast<int32_t>(cp);
    a.chunks = static_cast<int32_t>(max_blocks > 0 ? (max_blocks + cp - 1) / cp : 1);
    a.scores = scores;
    a.score_stride = score_stride;
    a.status = dev_status;
    return launch_status(launch_msa_scores(key_map, q_map, a, num_groups, G, static_cast<cudaStream_t>(stream)));
}

int dsa_msa_select(const float *scores, int64_t score_stride, const int32_t *row_ctx, int32_t num_rows,
                   int32_t max_ctx, int32_t *blocks, int32_t *dev_status, void *stream) {
    if (num_rows < 0 || max_ctx < 0) return DSA_ERR_INVALID_ARG;
    if (num_rows == 0) return DSA_OK;
    if (!scores || !row_ctx || !blocks) return DSA_ERR_INVALID_ARG;
    const int64_t max_blocks = (static_cast<int64_t>(max_ctx) + DSA_MSA_PAGE - 1) / DSA_MSA_PAGE;
    if (score_stride < max_blocks) return DSA_ERR_INVALID_ARG;
    if (max_blocks > 16384) return DSA_ERR_UNSUPPORTED;  // candidate keys live in shared memory
    MsaSelectArgs a;
    a.scores = scores;
    a.score_stride = score_stride;
    a.row_ctx = row_ctx;
    a.max_ctx = max_ctx;
    a.blocks = blocks;
    a.status = dev_status;
    return launch_status(launch_msa_select(a, num_rows, static_cast<cudaStream_t>(stream)));
}

size_t dsa_msa_attention_workspace_size(int32_t num_rows, int32_t heads_per_group) {
    if (num_rows <= 0 || heads_per_group <= 0) return 0;
    return msa_attention_workspace_bytes(static_cast<size_t>(num_rows), static_cast<size_t>(heads_per_group));
}

int dsa_msa_attention(const void *kv_pool, int64_t num_pages, float k_scale, float v_scale, const dsa_rows *rows,
                      const uint8_t *q, float q_scale, int32_t heads_per_group, const int32_t *blocks, float sm_scale,
                      float *out, float *lse, void *workspace, size_t workspace_bytes, int32_t *dev_status,
                      void *stream) {
    int rc = msa_check_rows(rows);
    if (rc != DSA_OK || rows->num_rows == 0) return rc;
    const int hpg = heads_per_group;
    if (hpg < 16 || hpg > DSA_MSA_MAX_HPG || hpg % 16 != 0) return DSA_ERR_UNSUPPORTED;
    if (!kv_pool || num_pages <= 0 || !q || !blocks || !out) return DSA_ERR_INVALID_ARG;
    if (!aligned(kv_pool, 16) || !aligned(q, 16)) return DSA_ERR_INVALID_ARG;
    for (float v : {k_scale, v_scale, q_scale, sm_scale})
        if (!std::isfinite(v) || !(v > 0.f)) return DSA_ERR_INVALID_ARG;
    const size_t need = msa_attention_workspace_bytes(static_cast<size_t>(rows->num_rows), static_cast<size_t>(hpg));
    if (workspace == nullptr || workspace_bytes < need) return DSA_ERR_WORKSPACE;
    if (!aligned(workspace, 256)) return DSA_ERR_INVALID_ARG;
    const uint64_t kv_rows = static_cast<uint64_t>(num_pages) * DSA_MSA_GROUPS * 2 * DSA_MSA_PAGE;
    if (kv_rows >= (1ull << 31)) return DSA_ERR_UNSUPPORTED;
    CUtensorMap kv_map, q_map;
    if (!encode_rows128(&kv_map, kv_pool, kv_rows, DSA_MSA_PAGE)) return DSA_ERR_CUDA;
    if (!encode_rows128(&q_map, q, static_cast<uint64_t>(rows->num_rows) * DSA_MSA_GROUPS * hpg,
                        static_cast<uint32_t>(hpg)))
        return DSA_ERR_CUDA;
    const size_t parts = static_cast<size_t>(rows->num_rows) * DSA_MSA_GROUPS * DSA_MSA_BLOCKS * hpg;
    MsaAttnArgs a;
    a.num_pages = num_pages;
    a.block_table = rows->block_table;
    a.bt_stride = rows->bt_stride;
    a.num_requests = rows->num_requests;
    a.row_req = rows->row_req;
    a.row_ctx = rows->row_ctx;
    a.max_ctx = rows->max_ctx;
    a.heads_per_group = hpg;
    a.blocks = blocks;
    a.s_scale = static_cast<float>(static_cast<double>(sm_scale) * q_scale * k_scale * 1.4426950408889634);
    a.v_scale = v_scale;
    a.part_o = static_cast<float *>(workspace);
    a.part_ml = reinterpret_cast<float *>(static_cast<uint8_t *>(workspace) +
                                          (parts * DSA_MSA_DIM * sizeof(float) + 255) / 256 * 256);
    a.out = out;
    a.lse = lse;
    a.status = dev_status;
    return launch_status(launch_msa_attention(kv_map, q_map, a, rows->num_rows, static_cast<cudaStream_t>(stream)));
}

// ------------------------------------------------------------------ dense K/V path

int dsa_rope_frequencies(int32_t rot_dim, double theta, int32_t scaling, double factor, int32_t trained_ctx,
                         double *inv_freq, float *scale) {
    if (rot_dim < 2 || rot_dim % 2 != 0 || inv_freq == nullptr || scale == nullptr) return DSA_ERR_INVALID_ARG;
    if (rot_dim > DSA_ROPE_MAX_DIM) return DSA_ERR_UNSUPPORTED;
    if (!std::isfinite(theta) || !(theta > 1.0)) return DSA_ERR_INVALID_ARG;
    if (scaling < DSA_ROPE_SCALE_NONE || scaling > DSA_ROPE_SCALE_YARN) return DSA_ERR_UNSUPPORTED;
    if (scaling != DSA_ROPE_SCALE_NONE && (!std::isfinite(factor) || !(factor >= 1.0))) return DSA_ERR_INVALID_ARG;
    if (scaling == DSA_ROPE_SCALE_YARN && trained_ctx < 1) return DSA_ERR_INVALID_ARG;
    const double base = scaling == DSA_ROPE_SCALE_NTK
                            ? theta * std::pow(factor, static_cast<double>(rot_dim) / (rot_dim > 2 ? rot_dim - 2 : 1))
                            : theta;
    if (!std::isfinite(base)) return DSA_ERR_INVALID_ARG;
    double lo = 0.0, hi = 0.0;
    if (scaling == DSA_ROPE_SCALE_YARN) {
        auto pair_of = [&](double turns) {
            return rot_dim * std::log(trained_ctx / (turns * 2.0 * M_PI)) / (2.0 * std::log(theta));
        };
        lo = std::fmax(std::floor(pair_of(32.0)), 0.0);
        hi = std::fmin(std::ceil(pair_of(1.0)), static_cast<double>(rot_dim - 1));
    }
    for (int i = 0; i < rot_dim / 2; ++i) {
        const double f = std::pow(base, -2.0 * i / rot_dim);
        if (scaling == DSA_ROPE_SCALE_LINEAR) {
            inv_freq[i] = f / factor;
        } else if (scaling == DSA_ROPE_SCALE_YARN) {
            const double r = std::fmin(std::fmax((i - lo) / std::fmax(hi - lo, 0.001), 0.0), 1.0);
            inv_freq[i] = f * (1.0 - r) + f / factor * r;
        } else {
            inv_freq[i] = f;
        }
    }
    *scale = scaling == DSA_ROPE_SCALE_YARN ? static_cast<float>(0.1 * std::log(factor) + 1.0) : 1.0f;
    return DSA_OK;
}

int dsa_rope_turns(const double *inv_freq, int32_t num_pairs, uint64_t *turns) {
    if (num_pairs < 0) return DSA_ERR_INVALID_ARG;
    if (num_pairs > 0 && (inv_freq == nullptr || turns == nullptr)) return DSA_ERR_INVALID_ARG;
    for (int i = 0; i < num_pairs; ++i)
        if (!std::isfinite(inv_freq[i])) return DSA_ERR_INVALID_ARG;
    for (int i = 0; i < num_pairs; ++i) {
        double x = inv_freq[i] / (2.0 * M_PI);
        x -= std::floor(x);  // in [0, 1]: a tiny negative angle can round to a whole turn
        turns[i] = x < 1.0 ? static_cast<uint64_t>(std::ldexp(x, 64)) : 0;
    }
    return DSA_OK;
}

static int check_rope_spec(const dsa_rope_spec *rope) {
    if (rope == nullptr || rope->turns == nullptr || rope->positions == nullptr) return DSA_ERR_INVALID_ARG;
    if (rope->rot_dim < 2 || rope->rot_dim % 2 != 0 || !std::isfinite(rope->scale)) return DSA_ERR_INVALID_ARG;
    return rope->rot_dim > DSA_ROPE_MAX_DIM ? DSA_ERR_UNSUPPORTED : DSA_OK;
}

extern "C++" {
// The angles of a call as the kernels take them.
static int rope_angles(const dsa_rope_spec *rope, RopeArgs *a) {
    const int rc = check_rope_spec(rope);
    if (rc != DSA_OK) return rc;
    a->turns = rope->turns;
    a->positions = rope->positions;
    a->rot = rope->rot_dim;
    a->scale = rope->scale;
    return DSA_OK;
}

static int rope_angles(const dsa_rope_axes *rope, RopeArgs *a) {
    if (rope == nullptr) return DSA_ERR_INVALID_ARG;
    const dsa_rope_spec one = {rope->turns, rope->positions, rope->rot_dim, rope->scale};
    const int rc = rope_angles(&one, a);
    if (rc != DSA_OK) return rc;
    if (rope->axis == nullptr || rope->num_axes < 1 || rope->axis_stride < 0) return DSA_ERR_INVALID_ARG;
    if (rope->num_axes > DSA_ROPE_MAX_AXES) return DSA_ERR_UNSUPPORTED;
    a->num_axes = rope->num_axes;
    a->axis_stride = rope->axis_stride;
    for (int p = 0; p < rope->rot_dim / 2; ++p) {
        if (rope->axis[p] >= rope->num_axes) return DSA_ERR_INVALID_ARG;
        a->axis[p >> 4] |= static_cast<uint32_t>(rope->axis[p]) << 2 * (p & 15);
    }
    return DSA_OK;
}
}  // extern "C++"

int dsa_rope_sections(const int32_t *sections, int32_t num_axes, int32_t order, int32_t num_pairs, uint8_t *axis) {
    if (num_axes > DSA_ROPE_MAX_AXES || num_pairs > DSA_ROPE_MAX_DIM / 2) return DSA_ERR_UNSUPPORTED;
    if (order != DSA_ROPE_AXES_SPLIT && order != DSA_ROPE_AXES_CYCLE) return DSA_ERR_UNSUPPORTED;
    if (sections == nullptr || axis == nullptr || num_axes < 1 || num_pairs < 1) return DSA_ERR_INVALID_ARG;
    int32_t left[DSA_ROPE_MAX_AXES] = {};
    int64_t total = 0;
    for (int x = 0; x < num_axes; ++x) {
        if (sections[x] < 0) return DSA_ERR_INVALID_ARG;
        total += left[x] = sections[x];
    }
    if (total != num_pairs) return DSA_ERR_INVALID_ARG;
    for (int p = 0, x = 0; p < num_pairs; ++p) {
        while (left[x] == 0) x = x + 1 < num_axes ? x + 1 : 0;
        axis[p] = static_cast<uint8_t>(x);
        --left[x];
        if (order == DSA_ROPE_AXES_CYCLE) x = x + 1 < num_axes ? x + 1 : 0;
    }
    return DSA_OK;
}

// Whether no two (token, head) parts of rot elements share an element: one of the strides steps over all of the
// other's.
static bool apart(int64_t token_stride, int64_t tokens, int64_t head_stride, int64_t heads, int64_t rot) {
    if (heads == 1) return tokens == 1 || token_stride >= rot;
    if (tokens == 1) return head_stride >= rot;
    return (head_stride >= rot && (token_stride - rot) / (heads - 1) >= head_stride) ||
           (token_stride >= rot && (head_stride - rot) / (tokens - 1) >= token_stride);
}

// Memory that a tensor takes: `width` bytes at base + t * token + h * head.
struct Span {
    uintptr_t base;
    int64_t tokens, token, heads, head, width;
    int64_t row() const { return (heads - 1) * head + width; }  // from a token's first byte to its last
};

// Whether the heads of two tokens meet, the second's first head `off` bytes behind the first's.
static bool rows_meet(const Span &a, const Span &b, int64_t off) {
    for (int64_t i = 0, j = 0; i < a.heads && j < b.heads;) {
        if (i * a.head + a.width <= off + j * b.head) ++i;
        else if (off + j * b.head + b.width <= i * a.head) ++j;
        else return true;
    }
    return false;
}

// Whether two tensors are known to share a byte: of tokens that follow one another (no token begins before the one
// before it ends) at one distance, or of a single token, that is decided; other layouts that lie within each other's
// range are left to the caller.
static bool meet(const Span &a, const Span &b) {
    const uintptr_t a_end = a.base + static_cast<uintptr_t>((a.tokens - 1) * a.token + a.row());
    const uintptr_t b_end = b.base + static_cast<uintptr_t>((b.tokens - 1) * b.token + b.row());
    if (a_end <= b.base || b_end <= a.base) return false;
    const int64_t d = static_cast<int64_t>(b.base - a.base);
    if (a.tokens == 1 && b.tokens == 1) return rows_meet(a, b, d);
    const int64_t step = a.tokens == 1 ? b.token : a.token;
    if ((a.tokens > 1 && b.tokens > 1 && a.token != b.token) || step < a.row() || step < b.row()) return false;
    // tokens whose numbers differ by q lie `off` apart, those one further off - step
    const int64_t q = d >= 0 ? d / step : -((-d + step - 1) / step), off = d - q * step;
    return (q < a.tokens && -q < b.tokens && rows_meet(a, b, off)) ||
           (q + 1 < a.tokens && -(q + 1) < b.tokens && rows_meet(a, b, off - step));
}

// Whether some token's row reaches into a block of memory.
static bool within(const Span &a, const Span &block) {
    const int64_t lo = static_cast<int64_t>(block.base - a.base) - a.row(), hi = lo + a.row() + block.width;
    if (hi <= 0) return false;             // token t does where lo < t * a.token < hi
    if (lo < 0 || a.tokens == 1 || a.token == 0) return lo < 0;
    const int64_t t = lo / a.token + 1;
    return t < a.tokens && t * a.token < hi;
}

static Span input_of(const RopeTensor &t, int32_t tokens, int32_t rot, int elem) {
    return {reinterpret_cast<uintptr_t>(t.x), tokens, t.x_token * elem, t.heads, t.x_head * elem, rot * elem};
}
static Span output_of(const RopeTensor &t, int32_t tokens, int32_t rot, int elem) {
    return {reinterpret_cast<uintptr_t>(t.out), tokens, t.out_token * elem, t.heads, t.out_head * elem, rot * elem};
}

// One rotated tensor, and whether 16-byte accesses reach all of its rotary parts.
static int rope_tensor(const dsa_rope_tensor &t, int32_t tokens, int32_t rot, int elem, RopeTensor *out) {
    if (t.x == nullptr || t.out == nullptr || t.num_heads < 1) return DSA_ERR_INVALID_ARG;
    if (t.layout != DSA_ROPE_INTERLEAVED && t.layout != DSA_ROPE_HALF) return DSA_ERR_UNSUPPORTED;
    if (t.num_heads > kRopeMaxHeads) return DSA_ERR_UNSUPPORTED;
    if (!aligned(t.x, elem) || !aligned(t.out, elem)) return DSA_ERR_INVALID_ARG;
    if (t.x == t.out && (t.x_token_stride != t.out_token_stride || t.x_head_stride != t.out_head_stride))
        return DSA_ERR_INVALID_ARG;
    if (t.x_token_stride < 0 || t.x_head_stride < 0 || t.out_token_stride < 0 || t.out_head_stride < 0)
        return DSA_ERR_INVALID_ARG;
    if (!apart(t.out_token_stride, tokens, t.out_head_stride, t.num_heads, rot)) return DSA_ERR_INVALID_ARG;
    const bool half = t.layout == DSA_ROPE_HALF;
    const int64_t v = 16 / elem;
    const bool vec = aligned(t.x, 16) && aligned(t.out, 16) && (half ? rot / 2 : rot) % v == 0 &&
                     t.x_token_stride % v == 0 && t.x_head_stride % v == 0 && t.out_token_stride % v == 0 &&
                     t.out_head_stride % v == 0;
    *out = RopeTensor{t.x, t.out, t.num_heads, half, vec, t.x_token_stride, t.x_head_stride, t.out_token_stride,
                      t.out_head_stride};
    if (t.x != t.out && meet(input_of(*out, tokens, rot, elem), output_of(*out, tokens, rot, elem)))
        return DSA_ERR_INVALID_ARG;
    return DSA_OK;
}

extern "C++" {
template <typename Spec>
static int rope_call(const Spec *rope, const dsa_rope_tensor *tensors, int32_t num_tensors, int32_t dtype,
                     int32_t num_tokens, void *stream) {
    if (num_tokens < 0 || num_tensors < 1) return DSA_ERR_INVALID_ARG;
    if (num_tensors > DSA_ROPE_MAX_TENSORS) return DSA_ERR_UNSUPPORTED;
    if (dtype != DSA_DTYPE_BF16 && dtype != DSA_DTYPE_FP32) return DSA_ERR_UNSUPPORTED;
    if (num_tokens == 0) return DSA_OK;
    RopeArgs a = {};
    int rc = rope_angles(rope, &a);
    if (rc != DSA_OK) return rc;
    if (tensors == nullptr) return DSA_ERR_INVALID_ARG;
    a.num_tokens = num_tokens;
    a.num_tensors = num_tensors;
    const int elem = dtype == DSA_DTYPE_BF16 ? 2 : 4;
    for (int i = 0; i < num_tensors; ++i) {
        rc = rope_tensor(tensors[i], num_tokens, rope->rot_dim, elem, &a.t[i]);
        if (rc != DSA_OK) return rc;
        const Span out = output_of(a.t[i], num_tokens, rope->rot_dim, elem);
        const Span x = input_of(a.t[i], num_tokens, rope->rot_dim, elem);
        for (int j = 0; j < i; ++j) {
            const Span other = output_of(a.t[j], num_tokens, rope->rot_dim, elem);
            if (a.t[i].out == a.t[j].out || a.t[i].out == a.t[j].x || a.t[i].x == a.t[j].out || meet(out, other) ||
                meet(x, other) || meet(out, input_of(a.t[j], num_tokens, rope->rot_dim, elem)))
                return DSA_ERR_INVALID_ARG;
        }
    }
    return launch_status(launch_rope(a, dtype, static_cast<cudaStream_t>(stream)));
}
}  // extern "C++"

int dsa_rope(const dsa_rope_spec *rope, const dsa_rope_tensor *tensors, int32_t num_tensors, int32_t dtype,
             int32_t num_tokens, void *stream) {
    return rope_call(rope, tensors, num_tensors, dtype, num_tokens, stream);
}

int dsa_rope_with_axes(const dsa_rope_axes *rope, const dsa_rope_tensor *tensors, int32_t num_tensors, int32_t dtype,
                       int32_t num_tokens, void *stream) {
    return rope_call(rope, tensors, num_tensors, dtype, num_tokens, stream);
}

// Geometry and address of a K/V pool.
static int check_kv_cache(const dsa_kv_cache *c) {
    if (c == nullptr) return DSA_ERR_INVALID_ARG;
    if (c->format != DSA_KV_BF16 && c->format != DSA_KV_FP8) return DSA_ERR_UNSUPPORTED;
    if (c->page_size != 16 && c->page_size != 32 && c->page_size != 64 && c->page_size != 128)
        return DSA_ERR_UNSUPPORTED;
    if (c->head_dim != 64 && c->head_dim != 128) return DSA_ERR_UNSUPPORTED;
    if (c->kv_heads < 1 || c->num_pages <= 0) return DSA_ERR_INVALID_ARG;
    if (c->kv_heads > kKvMaxHeads) return DSA_ERR_UNSUPPORTED;
    if (c->num_pages > ((1ll << 31) - 1) / (2ll * c->kv_heads * c->page_size)) return DSA_ERR_UNSUPPORTED;
    if (c->format == DSA_KV_FP8)
        for (float v : {c->k_scale, c->v_scale})
            if (!std::isfinite(v) || !(v > 0.f)) return DSA_ERR_INVALID_ARG;
    return DSA_OK;
}

extern "C++" {
template <typename Spec>
static int insert_call(const dsa_kv_cache *cache, const int32_t *slots, int32_t num_tokens, const dsa_kv_rows *kv,
                       const Spec *rope, const dsa_rope_tensor *q, int32_t *dev_status, void *stream) {
    int rc = check_kv_cache(cache);
    if (rc != DSA_OK) return rc;
    if (num_tokens < 0) return DSA_ERR_INVALID_ARG;
    if (num_tokens == 0) return DSA_OK;
    if (!cache->base || !aligned(cache->base, 16) || !slots || !kv || !kv->k || !kv->v) return DSA_ERR_INVALID_ARG;
    const int64_t width = static_cast<int64_t>(cache->kv_heads) * cache->head_dim;
    if (kv->k_stride < width || kv->v_stride < width) return DSA_ERR_INVALID_ARG;
    if (!aligned(kv->k, 2) || !aligned(kv->v, 2)) return DSA_ERR_INVALID_ARG;
    if (q != nullptr && rope == nullptr) return DSA_ERR_INVALID_ARG;
    KvInsertArgs a = {};
    a.rope.num_tokens = num_tokens;
    if (rope != nullptr) {
        rc = rope_angles(rope, &a.rope);
        if (rc != DSA_OK) return rc;
        if (kv->rot_offset < 0 || kv->rot_offset > cache->head_dim - rope->rot_dim) return DSA_ERR_INVALID_ARG;
        if (kv->layout != DSA_ROPE_INTERLEAVED && kv->layout != DSA_ROPE_HALF) return DSA_ERR_UNSUPPORTED;
        a.rot_offset = kv->rot_offset;
        a.half = kv->layout == DSA_ROPE_HALF;
        if (q != nullptr) {
            a.rope.num_tensors = 1;
            rc = rope_tensor(*q, num_tokens, rope->rot_dim, 2, &a.rope.t[0]);
            if (rc != DSA_OK) return rc;
            const Span out = output_of(a.rope.t[0], num_tokens, rope->rot_dim, 2);
            const Span k = {reinterpret_cast<uintptr_t>(kv->k), num_tokens, kv->k_stride * 2, 1, 0, width * 2};
            const Span v = {reinterpret_cast<uintptr_t>(kv->v), num_tokens, kv->v_stride * 2, 1, 0, width * 2};
            const Span pool = {reinterpret_cast<uintptr_t>(cache->base), 1, 0, 1, 0,
                               cache->num_pages * cache->page_size * 2 * width * (cache->format == DSA_KV_FP8 ? 1 : 2)};
            if (meet(out, k) || meet(out, v) || within(out, pool)) return DSA_ERR_INVALID_ARG;
        }
    }
    // 16-byte pieces need aligned rows, and rotary parts (or halves) of whole pieces
    a.vec = aligned(kv->k, 16) && aligned(kv->v, 16) && kv->k_stride % 8 == 0 && kv->v_stride % 8 == 0 &&
            a.rot_offset % 8 == 0 && a.rope.rot % (a.half ? 16 : 8) == 0;
    a.pool = static_cast<uint8_t *>(cache->base);
    a.fp8 = cache->format == DSA_KV_FP8;
    a.page_size = cache->page_size;
    for (a.page_shift = 4; 1 << a.page_shift < a.page_size;) ++a.page_shift;
    a.num_slots = cache->num_pages * cache->page_size;
    a.kv_heads = cache->kv_heads;
    a.head_dim = cache->head_dim;
    a.k_scale = cache->k_scale;
    a.v_scale = cache->v_scale;
    // (the reciprocals serve where neither they nor the remainders leave fp32's normal range)
    auto inverse = [](float s) { return s > 1e-20f && s < 1e20f ? static_cast<float>(1.0 / static_cast<double>(s)) : 0.f; };
    a.k_inv = inverse(cache->k_scale);
    a.v_inv = inverse(cache->v_scale);
    a.slots = slots;
    a.k = kv->k;
    a.v = kv->v;
    a.k_stride = kv->k_stride;
    a.v_stride = kv->v_stride;
    a.status = dev_status;
    return launch_status(launch_kv_insert(a, static_cast<cudaStream_t>(stream)));
}
}  // extern "C++"

int dsa_kv_insert(const dsa_kv_cache *cache, const int32_t *slots, int32_t num_tokens, const dsa_kv_rows *kv,
                  const dsa_rope_spec *rope, const dsa_rope_tensor *q, int32_t *dev_status, void *stream) {
    return insert_call(cache, slots, num_tokens, kv, rope, q, dev_status, stream);
}

int dsa_kv_insert_with_axes(const dsa_kv_cache *cache, const int32_t *slots, int32_t num_tokens, const dsa_kv_rows *kv,
                            const dsa_rope_axes *rope, const dsa_rope_tensor *q, int32_t *dev_status, void *stream) {
    return insert_call(cache, slots, num_tokens, kv, rope, q, dev_status, stream);
}

size_t dsa_kv_attention_workspace_size(const dsa_kv_cache *cache, int32_t num_rows, int32_t num_heads,
                                       int32_t max_ctx) {
    if (check_kv_cache(cache) != DSA_OK || num_rows <= 0 || num_heads <= 0 || max_ctx <= 0) return 0;
    if (max_ctx > DSA_KV_MAX_CTX) return 0;
    return kv_attention_workspace_bytes(num_rows, num_heads, cache->kv_heads, cache->head_dim, max_ctx);
}

// segments: NULL, or with one segment at least.
static int attention_call(const dsa_kv_cache *cache, const dsa_rows *rows, const dsa_kv_segments *segments,
                          const uint16_t *q, int64_t q_stride, int32_t num_heads, float sm_scale, uint16_t *out,
                          float *lse, void *workspace, size_t workspace_bytes, int32_t *dev_status, void *stream) {
    int rc = check_kv_cache(cache);
    if (rc != DSA_OK) return rc;
    if (rows == nullptr || rows->num_rows < 0 || rows->max_ctx < 0 || rows->num_requests < 0)
        return DSA_ERR_INVALID_ARG;
    const int G = rows->rows_per_group;
    if (G != 1 && G != 2 && G != 4 && G != 8) return DSA_ERR_UNSUPPORTED;
    if (num_heads < 1 || num_heads % cache->kv_heads != 0 || rows->num_rows % G != 0) return DSA_ERR_INVALID_ARG;
    if (num_heads / cache->kv_heads > DSA_KV_MAX_HPG || rows->max_ctx > DSA_KV_MAX_CTX) return DSA_ERR_UNSUPPORTED;
    if (!std::isfinite(sm_scale) || !(sm_scale > 0.f)) return DSA_ERR_INVALID_ARG;
    if (rows->num_rows == 0) return DSA_OK;
    if (!rows->block_table || !rows->row_req || !rows->row_ctx || !q || !out) return DSA_ERR_INVALID_ARG;
    if (!cache->base || !aligned(cache->base, 16) || !aligned(q, 16) || !aligned(out, 16)) return DSA_ERR_INVALID_ARG;
    if (q_stride < static_cast<int64_t>(num_heads) * cache->head_dim || q_stride % 8 != 0) return DSA_ERR_INVALID_ARG;
    const int64_t need_pages = (static_cast<int64_t>(rows->max_ctx) + cache->page_size - 1) / cache->page_size;
    if (rows->bt_stride < need_pages) return DSA_ERR_INVALID_ARG;
    if (segments != nullptr && (!segments->first_row || !segments->shared_ctx)) return DSA_ERR_INVALID_ARG;
    const size_t need = segments == nullptr
                            ? kv_attention_workspace_bytes(rows->num_rows, num_heads, cache->kv_heads, cache->head_dim,
                                                           rows->max_ctx)
                            : kv_attention_shared_workspace_bytes(rows->num_rows, num_heads, cache->kv_heads,
                                                                  cache->head_dim, rows->max_ctx, segments->num_segments,
                                                                  cache->format == DSA_KV_FP8);
    if (need > 0) {
        if (workspace == nullptr || workspace_bytes < need) return DSA_ERR_WORKSPACE;
        if (!aligned(workspace, 256)) return DSA_ERR_INVALID_ARG;
    }
    const int64_t row = static_cast<int64_t>(num_heads) * cache->head_dim * 2;
    const Span q_span = {reinterpret_cast<uintptr_t>(q), rows->num_rows, q_stride * 2, 1, 0, row};
    const Span out_span = {reinterpret_cast<uintptr_t>(out), 1, 0, 1, 0, rows->num_rows * row};
    const Span lse_span = {reinterpret_cast<uintptr_t>(lse), 1, 0, 1, 0, static_cast<int64_t>(rows->num_rows) * num_heads * 4};
    if (within(q_span, out_span) || (lse != nullptr && (within(q_span, lse_span) || within(out_span, lse_span))))
        return DSA_ERR_INVALID_ARG;
    const bool fp8 = cache->format == DSA_KV_FP8;
    KvAttnArgs a = {};
    a.pool = cache->base;
    a.pool_rows = static_cast<uint64_t>(cache->num_pages) * cache->kv_heads * 2 * cache->page_size;
    a.fp8 = fp8;
    a.page_size = cache->page_size;
    a.num_pages = cache->num_pages;
    a.kv_heads = cache->kv_heads;
    a.head_dim = cache->head_dim;
    a.block_table = rows->block_table;
    a.bt_stride = rows->bt_stride;
    a.num_requests = rows->num_requests;
    a.row_req = rows->row_req;
    a.row_ctx = rows->row_ctx;
    a.num_rows = rows->num_rows;
    a.max_ctx = rows->max_ctx;
    a.group = G;
    a.q = q;
    a.q_stride = q_stride;
    a.num_heads = num_heads;
    a.s_scale = static_cast<float>(static_cast<double>(sm_scale) * (fp8 ? cache->k_scale : 1.0) * 1.4426950408889634);
    a.v_scale = fp8 ? cache->v_scale : 1.0f;
    a.out = out;
    a.lse = lse;
    a.status = dev_status;
    if (segments == nullptr) return launch_status(launch_kv_attention(a, workspace, static_cast<cudaStream_t>(stream)));
    const KvSegmentArgs seg = {segments->first_row, segments->shared_ctx, segments->num_segments, segments->least_saved};
    return launch_status(launch_kv_attention_shared(seg, a, workspace, static_cast<cudaStream_t>(stream)));
}

int dsa_kv_attention(const dsa_kv_cache *cache, const dsa_rows *rows, const uint16_t *q, int64_t q_stride,
                     int32_t num_heads, float sm_scale, uint16_t *out, float *lse, void *workspace,
                     size_t workspace_bytes, int32_t *dev_status, void *stream) {
    return attention_call(cache, rows, nullptr, q, q_stride, num_heads, sm_scale, out, lse, workspace, workspace_bytes,
                          dev_status, stream);
}

size_t dsa_kv_attention_shared_workspace_size(const dsa_kv_cache *cache, int32_t num_rows, int32_t num_heads,
                                              int32_t max_ctx, int32_t num_segments) {
    if (num_segments <= 0)
        return num_segments < 0 ? 0 : dsa_kv_attention_workspace_size(cache, num_rows, num_heads, max_ctx);
    if (check_kv_cache(cache) != DSA_OK || num_rows <= 0 || num_heads <= 0 || max_ctx <= 0) return 0;
    if (max_ctx > DSA_KV_MAX_CTX) return 0;
    return kv_attention_shared_workspace_bytes(num_rows, num_heads, cache->kv_heads, cache->head_dim, max_ctx,
                                               num_segments, cache->format == DSA_KV_FP8);
}

int dsa_kv_attention_shared(const dsa_kv_cache *cache, const dsa_rows *rows, const dsa_kv_segments *segments,
                            const uint16_t *q, int64_t q_stride, int32_t num_heads, float sm_scale, uint16_t *out,
                            float *lse, void *workspace, size_t workspace_bytes, int32_t *dev_status, void *stream) {
    if (segments == nullptr || segments->num_segments < 0 || segments->least_saved < 0) return DSA_ERR_INVALID_ARG;
    const bool some = segments->num_segments > 0 && rows != nullptr && rows->max_ctx > 0;
    return attention_call(cache, rows, some ? segments : nullptr, q, q_stride, num_heads, sm_scale, out, lse, workspace,
                          workspace_bytes, dev_status, stream);
}

int dsa_kv_plan(const dsa_kv_step *step, int32_t *dev_status, void *stream) {
    if (step == nullptr) return DSA_ERR_INVALID_ARG;
    const dsa_kv_step &p = *step;
    if (p.page_size != 16 && p.page_size != 32 && p.page_size != 64 && p.page_size != 128) return DSA_ERR_UNSUPPORTED;
    if (p.rows_per_group != 1 && p.rows_per_group != 2 && p.rows_per_group != 4 && p.rows_per_group != 8)
        return DSA_ERR_UNSUPPORTED;
    if (p.num_requests < 0 || p.num_pages < 0 || p.bt_stride < 0 || p.free_capacity < 0 || p.num_segments < 0 ||
        p.max_rows < 0 || p.max_rows % p.rows_per_group != 0)
        return DSA_ERR_INVALID_ARG;
    if (p.num_requests > DSA_KV_PLAN_MAX_REQUESTS || p.num_pages > ((1ll << 31) - 1) / p.page_size)
        return DSA_ERR_UNSUPPORTED;
    if (p.free_count == nullptr || (p.free_capacity > 0 && p.free_pages == nullptr)) return DSA_ERR_INVALID_ARG;
    if (p.num_requests > 0 && (!p.context || !p.new_tokens || (p.bt_stride > 0 && !p.block_table)))
        return DSA_ERR_INVALID_ARG;
    if (p.max_rows > 0 && (!p.row_req || !p.row_ctx)) return DSA_ERR_INVALID_ARG;
    if (p.num_segments > 0 && (!p.segment_requests || !p.segment_rows)) return DSA_ERR_INVALID_ARG;
    if (p.bt_stride > (1ll << 31)) return DSA_ERR_UNSUPPORTED;
    // what a call writes lies apart from all else that it touches
    struct Block {
        const void *base;
        int64_t words;
        bool written;
    };
    const int64_t n = p.num_requests, rows = p.max_rows, segs = p.num_segments > 0 ? p.num_segments + 1ll : 0;
    const bool same_context = p.context_out == p.context, same_count = p.free_count_out == p.free_count;
    const Block blocks[] = {{p.context, n, same_context}, {p.new_tokens, n, false}, {p.first_own, n, false},
                            {p.free_count, 1, same_count}, {p.segment_requests, segs, false},
                            {p.block_table, n * p.bt_stride, true}, {p.free_pages, p.free_capacity, true},
                            {p.row_req, rows, true}, {p.row_ctx, rows, true}, {p.positions, rows, true},
                            {p.slots, rows, true}, {p.row_start, n + 1, true}, {p.granted, n, true},
                            {same_context ? nullptr : p.context_out, n, true},
                            {same_count ? nullptr : p.free_count_out, 1, true},
                            {p.segment_rows, segs, true}, {dev_status, 1, true}};
    for (const Block &x : blocks) {
        if (x.base == nullptr || x.words == 0) continue;
        if (!aligned(x.base, 4)) return DSA_ERR_INVALID_ARG;
        for (const Block *y = blocks; y != &x; ++y) {
            if (y->base == nullptr || y->words == 0 || !(x.written || y->written)) continue;
            const uintptr_t a = reinterpret_cast<uintptr_t>(x.base), b = reinterpret_cast<uintptr_t>(y->base);
            if (a < b + static_cast<uintptr_t>(y->words) * 4 && b < a + static_cast<uintptr_t>(x.words) * 4)
                return DSA_ERR_INVALID_ARG;
        }
    }
    KvPlanArgs a = {};
    a.num_requests = p.num_requests;
    a.page_size = p.page_size;
    for (a.page_shift = 4; 1 << a.page_shift < a.page_size;) ++a.page_shift;
    a.num_pages = p.num_pages;
    const int64_t most = p.bt_stride * p.page_size;
    a.capacity = most < 0x7fffffff ? static_cast<int32_t>(most) : 0x7fffffff;
    a.context = p.context;
    a.new_tokens = p.new_tokens;
    a.first_own = p.first_own;
    a.block_table = p.block_table;
    a.bt_stride = p.bt_stride;
    a.free_pages = p.free_pages;
    a.free_capacity = p.free_capacity;
    a.free_count = p.free_count;
    a.segment_requests = p.segment_requests;
    a.num_segments = p.num_segments;
    a.max_rows = p.max_rows;
    a.group = p.rows_per_group;
    a.row_req = p.row_req;
    a.row_ctx = p.row_ctx;
    a.positions = p.positions;
    a.slots = p.slots;
    a.row_start = p.row_start;
    a.granted = p.granted;
    a.context_out = p.context_out;
    a.free_count_out = p.free_count_out;
    a.segment_rows = p.segment_rows;
    a.status = dev_status;
    return launch_status(launch_kv_plan(a, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
