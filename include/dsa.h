/*
 * dsa.h -- C ABI of libdsa, a single-GPU (sm_103a) implementation of the
 * DeepSeek-style sparse attention (DSA) layer as used in Kimi K3.1 Pro.
 *
 * The layer (vLLM blog "Day-0 support for Kimi K3.1 Pro", section "Sparse
 * attention in K3.1 Pro", Fig. 1): for every query row a small indexer with
 * 32 FP8 heads scores every earlier token against that token's FP8 index key
 * (132 B with its scale); a top-k step keeps the 2,048 best tokens; exact
 * absorbed-MLA attention of 96 query heads then runs over only those tokens'
 * 576-byte latents (512 latent + 64 RoPE dims).  Both caches are paged and
 * are read through a block table that is translated to physical slots
 * before the attention step (section "One KV cache, three states"; in the
 * fused decode path the scorer and the top-k hand attention the physical
 * cache rows to read, section "Low-latency decode: fused DSA decode path").
 *
 * Conventions shared by every entry point
 *   - Every pointer argument is a DEVICE pointer owned by the caller, unless
 *     its comment says "host".  Struct arguments themselves are host memory
 *     and are read only during the call.  The library allocates no device
 *     memory and keeps no state between calls (per-device tensor-map encoder
 *     lookup aside).
 *   - `stream` is a cudaStream_t passed as void*; NULL means the legacy
 *     default stream.  Every call only enqueues work and returns; nothing
 *     synchronises with the host.
 *   - The int return value is a host-side status: arguments are checked
 *     before anything is launched, and a launch error is reported as
 *     DSA_ERR_CUDA.  No exceptions cross the boundary.
 *   - Errors the kernels find in device data (a page id outside the pool, a
 *     context longer than max_ctx, a timed-out wait) are written to the
 *     optional `dev_status` word (int32, device memory): the first error
 *     code is kept (compare-and-swap from 0), later ones are dropped.  The
 *     caller zeroes it before the calls and reads it after synchronising.
 *     Outputs of a call that reported a device error are unspecified.
 *   - Results are deterministic, and a row's results do not depend on the
 *     other rows of the batch (batch invariance).
 *
 * Cache page layouts (page_size 64; the per-token widths are the blog's,
 * "One KV cache, three states": index key 132 B FP8 / 68 B MXFP4, latent
 * 576 B FP8 / 352 B NVFP4; the arrangement within a page is this library's):
 *   DSA_KEY_FP8      [64 x 128 B e4m3 key][64 x fp32 per-token scale]   8448 B
 *   DSA_KEY_MXFP4    [64 x 64 B e2m1 pairs][64 x 4 B e8m0, one per 32]  4352 B
 *   DSA_LATENT_FP8   [64 x 576 B e4m3], scale = dsa_cache.tensor_scale 36864 B
 *   DSA_LATENT_NVFP4 [64 x 256 B e2m1 pairs][64 x 32 B e4m3 scale, one per 16]
 *                    [64 x 64 B e4m3 RoPE dims, scale = tensor_scale]   22528 B
 * e2m1 pairs hold element 2j in the low nibble.  Token t of a request lives
 * in page block_table[req][t / 64], row t % 64; its physical slot is
 * page * 64 + t % 64, the same slot id in the index and the latent pool.
 */
#ifndef DSA_H_
#define DSA_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* ---- status codes */
#define DSA_OK 0
#define DSA_ERR_INVALID_ARG (-1)  /* host: null pointer, bad size or stride */
#define DSA_ERR_UNSUPPORTED (-2)  /* host: format, page size, head count or k not supported */
#define DSA_ERR_CUDA (-3)         /* host: a CUDA call or launch failed */
#define DSA_ERR_WORKSPACE (-4)    /* host: workspace smaller than dsa_*_workspace_size() */
#define DSA_ERR_TIMEOUT (-5)      /* device: a bounded wait inside a kernel gave up */
#define DSA_ERR_BOUNDS (-6)       /* device: page id, slot or context outside its range */
#define DSA_ERR_RANGE (-7)        /* device: a value the kernel cannot represent (e.g. |q| > 65504) */

/* ---- cache formats */
#define DSA_KEY_FP8 1
#define DSA_KEY_MXFP4 2
#define DSA_LATENT_FP8 3
#define DSA_LATENT_NVFP4 4

/* ---- fixed dimensions of the layer */
#define DSA_PAGE_SIZE 64
#define DSA_INDEX_HEADS 32
#define DSA_INDEX_DIM 128
#define DSA_LATENT_DIM 576 /* 512 latent + 64 RoPE dims */
#define DSA_VALUE_DIM 512
#define DSA_MAX_HEADS 128  /* MLA query heads per row, multiple of 16 */
#define DSA_MAX_TOPK 2048

/* One paged cache pool (index keys or latents). */
typedef struct dsa_cache {
    const void *base;     /* device, num_pages * page bytes, 16-byte aligned (DSA_KEY_MXFP4: 32-byte
                             aligned, the rule of the 4-bit tensor copies; else DSA_ERR_INVALID_ARG) */
    int32_t format;       /* DSA_KEY_* for an index pool, DSA_LATENT_* for a latent pool */
    int32_t page_size;    /* must be DSA_PAGE_SIZE */
    int64_t num_pages;
    float tensor_scale;   /* latent pools: per-tensor scale of the e4m3 codes; ignored for index pools */
} dsa_cache;

/* Query rows and their addressing. */
typedef struct dsa_rows {
    const int32_t *block_table; /* device [num_requests, bt_stride] physical page ids */
    int64_t bt_stride;          /* entries per request, >= ceil(max_ctx / 64) */
    int32_t num_requests;       /* rows of block_table; row_req outside [0, num_requests) is DSA_ERR_BOUNDS */
    const int32_t *row_req;     /* device [num_rows] request of each row */
    const int32_t *row_ctx;     /* device [num_rows] visible tokens L_r (positions 0..L_r-1, incl. itself) */
    int32_t num_rows;
    int32_t max_ctx;            /* host bound on every row_ctx; larger values are DSA_ERR_BOUNDS */
    int32_t rows_per_group;     /* 1, 2, 4 or 8: consecutive rows of one request that the indexer
                                   scores against one read of the keys (speculative-verify rows,
                                   prefill query blocks); num_rows must be a multiple of it */
} dsa_rows;

/*
 * Indexer logits (blog section "Sparse attention in K3.1 Pro"; the weighted,
 * fp32-accumulated reduction across heads is the AMD section "Quantization:
 * native MXFP4 indexer"; the query carries no scale because the head
 * weights are folded into its quantisation, section "Low-latency decode:
 * fused DSA decode path"):
 *
 *   logits[r * logits_stride + t] = sum_{h<32} head_w[r,h] * max(0, s_t * <q_idx[r,h,:], k_t>)
 *   for 0 <= t < row_ctx[r]
 *
 * k_t is token t's decoded key (e4m3 codes with s_t its fp32 scale, or
 * MXFP4 e2m1 * 2^(e8m0-127) with s_t = 1).  q_idx: [num_rows, 32, 128] e4m3
 * codes (16-byte aligned); head_w: [num_rows, 32] fp32; logits: fp32 with
 * row stride logits_stride >= max_ctx.  Entries at t >= row_ctx[r] are not
 * written.  Products are exact and accumulate in fp32 on the tensor cores,
 * so a logit differs from an exact evaluation by accumulation rounding only.
 * MXFP4 keys multiply their e2m1 codes by the block scales inside the MMA
 * (block-scaled e2m1 x e4m3); a visible key with the e8m0 NaN code 0xff is
 * DSA_ERR_RANGE (its logits are then unspecified).
 */
int dsa_indexer_logits(const dsa_cache *index_cache, const dsa_rows *rows, const uint8_t *q_idx,
                       const float *head_w, float *logits, int64_t logits_stride, int32_t *dev_status,
                       void *stream);

/*
 * Top-k (blog section "Sparse attention in K3.1 Pro": only the 2,048 best
 * scored tokens are kept; the fused path's selection is exact, section
 * "Low-latency decode"):
 *
 *   idx_out[r, 0..k) = the min(k, row_ctx[r]) positions t < row_ctx[r] with
 *   the largest logits[r * logits_stride + t], ties broken toward the lower t,
 *   written in ascending order of t and padded with -1.
 *
 * Logits compare as floats (-0 == +0); they must be finite.  k in
 * [1, DSA_MAX_TOPK].  Exact and deterministic: given identical logits the
 * result is bit-identical.
 *
 * workspace (device, 256-byte aligned, no initial contents) may be NULL.
 * With workspace_bytes >= dsa_topk_workspace_size(num_rows, max_ctx, k) > 0
 * (at most 64 rows, max_ctx above 131,072), the selection runs as three launches of
 * independent CTAs over chunks of each row: every chunk counts its keys in
 * 4096 bins (the top 12 bits of the order-preserving key: one bin per 1/8
 * binade); every chunk sums its row's counts, finds the bin holding the k-th
 * largest key and passes on its keys at or above that bin, in position order;
 * every chunk then finds the exact threshold among the row's keys in that bin
 * and writes its share of the selection.  A row whose threshold bin holds more
 * than 12,288 keys (heavy ties, or scores within 1/8 binade of each other) is
 * selected from its whole logits by one CTA instead (slower).  Without it
 * (NULL, or a size of 0 for this shape), one thread-block cluster per row
 * selects.  A workspace smaller than the size is DSA_ERR_WORKSPACE.  The
 * result is the same either way.
 */
int dsa_topk(const float *logits, int64_t logits_stride, const int32_t *row_ctx, int32_t num_rows,
             int32_t max_ctx, int32_t k, int32_t *idx_out, int32_t *dev_status, void *workspace,
             size_t workspace_bytes, void *stream);

/* Workspace bytes of the histogram top-k for this batch on the current device; 0 when the shape
 * (more than 64 rows, or rows of at most 131,072 keys) takes the cluster selection, which needs none. */
size_t dsa_topk_workspace_size(int32_t num_rows, int32_t max_ctx, int32_t k);

/*
 * Top-k and page -> slot in one call (the two steps below, dsa_topk then
 * dsa_page_to_slot, with the translation done where the selection is
 * written): idx_out as dsa_topk over rows->row_ctx / rows->max_ctx, and
 * slots_out[r, i] = block_table[row_req[r]][t / 64] * 64 + t % 64 for each
 * selected t = idx_out[r, i] (-1 where idx_out is -1).  A page id outside
 * [0, pool_pages) or a bad row_req is DSA_ERR_BOUNDS with slot -1.  workspace
 * as for dsa_topk.
 */
int dsa_topk_slots(const float *logits, int64_t logits_stride, const dsa_rows *rows, int64_t pool_pages, int32_t k,
                   int32_t *idx_out, int32_t *slots_out, int32_t *dev_status, void *workspace, size_t workspace_bytes,
                   void *stream);

/*
 * dsa_topk_slots whose output pass also warms L2 with the selected tokens'
 * latents, so that the sparse attention launched next gathers them from L2
 * instead of HBM (the fused decode path of blog section "Low-latency decode"
 * hands attention the physical rows to read as soon as they are chosen).
 * latent_cache: the latent pool the slots index (its num_pages bounds the
 * slots).  FP8 latents (576 contiguous bytes per slot) are prefetched; an
 * NVFP4 pool gets the plain dsa_topk_slots result.  Outputs are identical to
 * dsa_topk_slots.  workspace as for dsa_topk.
 */
int dsa_topk_slots_warm(const float *logits, int64_t logits_stride, const dsa_rows *rows, const dsa_cache *latent_cache,
                        int32_t k, int32_t *idx_out, int32_t *slots_out, int32_t *dev_status, void *workspace,
                        size_t workspace_bytes, void *stream);

/*
 * Single-pass scorer + top-k (blog section "Low-latency decode: fused DSA
 * decode path": the scorer feeds a batch-invariant exact top-k; here the
 * scorer's epilogue also builds the histogram the selection starts from).
 *
 * DSA_HIST_BINS bins per row of the top 16 bits of each logit's
 * order-preserving 32-bit key (larger float, larger key; -0 folds onto +0).
 *
 * dsa_indexer_logits_hist: dsa_indexer_logits, and for every logit it writes
 *   hist[r * DSA_HIST_BINS + (key(logit) >> 16)] += 1.
 *   hist: [num_rows, DSA_HIST_BINS] uint32, device, all zero on entry.
 *
 * dsa_topk_hist: dsa_topk (same arguments and result), starting from that
 *   histogram: the bin holding the k-th key is read off it, one pass over the
 *   logits collects that bin's keys, and the selection finishes on those.
 *   hist must be the histogram dsa_indexer_logits_hist produced for exactly
 *   these logits and row_ctx (otherwise the result is undefined); the call
 *   leaves it all zero, ready for the next scorer call.  A bin holding more
 *   keys than the candidate list falls back to refinement rounds.
 *
 * dsa_indexer_topk: both calls in one, with the logits and the histogram in
 *   a workspace of dsa_indexer_topk_workspace_size() bytes (device, 256-byte
 *   aligned) that must be all zero before the first call; every call leaves
 *   its histogram part zero again, and the logits part holds no defined
 *   contents afterwards (their L2 lines are dropped once read, so they cost no
 *   HBM write-back).
 */
#define DSA_HIST_BINS 65536
int dsa_indexer_logits_hist(const dsa_cache *index_cache, const dsa_rows *rows, const uint8_t *q_idx,
                            const float *head_w, float *logits, int64_t logits_stride, uint32_t *hist,
                            int32_t *dev_status, void *stream);
int dsa_topk_hist(const float *logits, int64_t logits_stride, const int32_t *row_ctx, int32_t num_rows,
                  int32_t max_ctx, int32_t k, uint32_t *hist, int32_t *idx_out, int32_t *dev_status, void *stream);
int dsa_indexer_topk(const dsa_cache *index_cache, const dsa_rows *rows, const uint8_t *q_idx, const float *head_w,
                     int32_t k, int32_t *idx_out, int32_t *dev_status, void *workspace, size_t workspace_bytes,
                     void *stream);
size_t dsa_indexer_topk_workspace_size(int32_t num_rows, int32_t max_ctx);

/*
 * Page -> slot translation (blog section "One KV cache, three states": the
 * block table and cache slots are translated to kernel page addresses
 * before each step):
 *
 *   slots[r, i] = block_table[row_req[r]][t / 64] * 64 + t % 64 for t = idx[r, i] >= 0,
 *   slots[r, i] = -1 for t = -1.
 *
 * idx and slots are [num_rows, k] int32.  A position t >= row_ctx[r], or a
 * page id outside [0, pool_pages) (the page count of the pools the slots
 * will address), is DSA_ERR_BOUNDS and yields slot -1.
 */
int dsa_page_to_slot(const dsa_rows *rows, int64_t pool_pages, const int32_t *idx, int32_t k, int32_t *slots,
                     int32_t *dev_status, void *stream);

/*
 * Sparse absorbed MLA (blog section "Sparse attention in K3.1 Pro": MLA
 * attention runs exactly, but only over the selected tokens; the latent is
 * both key and value, section "Low-latency decode": absorbed key
 * projection):
 *
 *   S[h, t] = sm_scale * <q[r,h,:], kv_t>                     (576 dims)
 *   out[r,h,:] = sum_t softmax_t(S[h, .]) * kv_t[0:512]      over t in slots[r, :] with slot >= 0
 *   lse[r,h] = ln sum_t exp(S[h,t])
 *
 * kv_t is the decoded latent of slot t (FP8: e4m3 * tensor_scale; NVFP4:
 * e2m1 * per-16 e4m3 scale for dims 0..511 and e4m3 * tensor_scale for the
 * RoPE dims).  q: [num_rows, num_heads, 576] bf16 bits, num_heads a multiple
 * of 16 and <= 96; slots: [num_rows, k] int32, -1 = unused; out:
 * [num_rows, num_heads, 512] fp32; lse: [num_rows, num_heads] fp32 or NULL.
 * A row with no valid slot gets out = 0 and lse = -inf.  Precision:
 *   - _decode over FP8 latents (k > 128) contracts e4m3 x e4m3 -> fp32 on the
 *     latents as stored.  Each head's query is scaled by a power of two and
 *     written as the sum of two e4m3 terms (exact for bf16 values within
 *     about 2^10 of the head's largest |q|; smaller ones keep an absolute
 *     error of at most 2^-17 of that largest), and the softmax weights likewise
 *     (about 8 significant bits).  A non-finite q is DSA_ERR_RANGE.
 *   - NVFP4 latents, _prefill, and decode with k <= 128 contract
 *     fp16 x fp16 -> fp32: latents decode to fp16 exactly, q rounds from bf16
 *     to fp16 (|q| > 65504 is DSA_ERR_RANGE), weights are fp16.
 *
 * _decode splits each row's k tokens into parts of 128 (k <= 2048, else
 * DSA_ERR_UNSUPPORTED), one CTA per part, keeps each part's normalised
 * output in fp16 and merges the parts by log-sum-exp; it needs a workspace
 * of dsa_sparse_mla_workspace_size() bytes (device, 256-byte aligned, no
 * initial contents; it also holds the rows' queries converted once to the
 * kernel's fp16 layout).  _prefill runs one CTA per row, needs no workspace
 * (pass NULL, 0) and suits many rows.  The split is fixed, so both are
 * batch-invariant; their results differ from each other by rounding.
 */
int dsa_sparse_mla_decode(const dsa_cache *latent_cache, const uint16_t *q, int32_t num_heads,
                          const int32_t *slots, int32_t num_rows, int32_t k, float sm_scale, float *out,
                          float *lse, int32_t *dev_status, void *workspace, size_t workspace_bytes, void *stream);

int dsa_sparse_mla_prefill(const dsa_cache *latent_cache, const uint16_t *q, int32_t num_heads,
                           const int32_t *slots, int32_t num_rows, int32_t k, float sm_scale, float *out,
                           float *lse, int32_t *dev_status, void *workspace, size_t workspace_bytes,
                           void *stream);

/*
 * dsa_sparse_mla_decode in two parts, so the query conversion can run ahead
 * of (or beside) the scorer and the top-k, which it does not depend on:
 * _prepare writes each row's query, converted once to the attention
 * kernel's fp16 operand layout, into the workspace (nothing when k <= 128,
 * where decode uses no workspace); _prepared then runs the attention on it.
 * Both take the arguments of dsa_sparse_mla_decode (_prepare ignores the
 * slots, outputs and sm_scale) and the same workspace; _prepared must be
 * ordered after _prepare with the same q, num_heads, num_rows and k.  The
 * result equals dsa_sparse_mla_decode's bit for bit.
 */
int dsa_sparse_mla_decode_prepare(const dsa_cache *latent_cache, const uint16_t *q, int32_t num_heads,
                                  int32_t num_rows, int32_t k, int32_t *dev_status, void *workspace,
                                  size_t workspace_bytes, void *stream);
int dsa_sparse_mla_decode_prepared(const dsa_cache *latent_cache, const uint16_t *q, int32_t num_heads,
                                   const int32_t *slots, int32_t num_rows, int32_t k, float sm_scale, float *out,
                                   float *lse, int32_t *dev_status, void *workspace, size_t workspace_bytes,
                                   void *stream);

/*
 * dsa_sparse_mla_decode without a caller workspace.  The paper has no
 * counterpart to this call; it exists for callers that cannot allocate
 * device memory: a host framework whose allocator has reserved the device's
 * memory for its own pools and hands out no extra buffers, a plugin that
 * only sees the tensors it is given, or a latency-critical loop that must not
 * call cudaMalloc (it can block and synchronise the device).
 *
 * Same arguments, semantics and results as dsa_sparse_mla_decode, minus the
 * workspace.  The split-K partial outputs live in a fixed array in the
 * library's own device memory, sized for DSA_NOALLOC_MAX_ROWS rows of
 * k <= 2048 tokens and num_heads <= 96 (13,569,024 bytes, held by every GPU
 * that loads the library until the process exits).  Larger calls return
 * DSA_ERR_WORKSPACE without launching.  The first call on a device looks up
 * the array's address with that device current; make it before capturing
 * any stream.  That address belongs to the device's primary context: after a
 * cudaDeviceReset of the device this call must not be used again in the
 * process.  Shape errors return the statuses dsa_sparse_mla_decode returns.  All calls share the array: calls whose kernels may overlap on
 * the GPU (unordered streams) race on it; calls ordered on one stream do not.
 * No part of the array needs to start zeroed.
 */
#define DSA_NOALLOC_MAX_ROWS 8
int dsa_sparse_mla_decode_noalloc(const dsa_cache *latent_cache, const uint16_t *q, int32_t num_heads,
                                  const int32_t *slots, int32_t num_rows, int32_t k, float sm_scale, float *out,
                                  float *lse, int32_t *dev_status, void *stream);

/*
 * Quantise new tokens and write them into the caches (blog section
 * "Low-latency decode: fused DSA decode path": the front end quantises the
 * new token's index key, FP8 or MXFP4, and the new latent is written into
 * the cache before the indexer scores).  For each i with slots[i] >= 0 the
 * token's index key index_keys[i, 0:128] (bf16 bits) and latent
 * latents[i, 0:576] (bf16 bits) are written at that physical slot of the two
 * pools (the pools' base pointers are written through):
 *   DSA_KEY_FP8:      s = amax / 448 (1 if amax = 0), code = e4m3(x / s), s stored as fp32
 *   DSA_KEY_MXFP4:    per 32 values E = floor(log2 amax) - 2 + 127 clamped to [0, 254]
 *                     (0 for an all-zero block), code = e2m1(x * 2^(127 - E))
 *   DSA_LATENT_FP8:   code = e4m3(x / tensor_scale)
 *   DSA_LATENT_NVFP4: per 16 values scale code = e4m3(amax / 6), code = e2m1(x / scale)
 *                     (0 when the scale is 0); RoPE dims e4m3(x / tensor_scale)
 * Scales and quotients are IEEE fp32 operations; codes are round-to-nearest-
 * even with saturation (e4m3 to +-448, e2m1 to +-6), so the bytes are exact.
 * Both pools must have the same num_pages; tensor_scale > 0 comes from the
 * latent pool.  A slot outside the pools is DSA_ERR_BOUNDS (not written).
 */
int dsa_cache_insert(const dsa_cache *index_cache, const dsa_cache *latent_cache, const int32_t *slots,
                     int32_t num_tokens, const uint16_t *index_keys, const uint16_t *latents, int32_t *dev_status,
                     void *stream);

/* Workspace bytes dsa_sparse_mla_decode needs for num_rows rows of k slots. */
size_t dsa_sparse_mla_workspace_size(int32_t num_rows, int32_t num_heads, int32_t k);

/*
 * ---- MSA, the block-sparse variant (vLLM blog "Day-0 support for
 * MiniMax-M3.1-Flash", section "MSA primer" and its Fig. 1; FP8 queries over an
 * FP8 K/V cache, section "Blackwell-optimised MSA kernels").  The cache is cut
 * into 128-token blocks, which are also its pages; one index query per GQA
 * group (4 groups = 4 KV heads) scores every visible token against the one
 * 128-B index key all groups share, the scores are max-pooled per block, each
 * group keeps its most recent block and the 15 best others, and the group's
 * query heads attend exactly to the tokens of those blocks.
 *
 * Page layouts (128 tokens; the widths are the blog's, the arrangement inside
 * a page is this library's):
 *   index  [128 x 128 B e4m3]                                          16384 B
 *   kv     [4 KV heads] x ([K: 128 x 128 B e4m3] [V: 128 x 128 B e4m3]) 131072 B
 * For these calls dsa_rows.block_table holds 128-token page ids (bt_stride >=
 * ceil(max_ctx / 128)); token t of a request is row t % 128 of page
 * block_table[req][t / 128].  Pools and queries are 16-byte aligned.
 */
#define DSA_MSA_PAGE 128
#define DSA_MSA_DIM 128
#define DSA_MSA_GROUPS 4
#define DSA_MSA_BLOCKS 16   /* blocks kept per (row, group): the most recent + the 15 best others */
#define DSA_MSA_MAX_HPG 64  /* query heads per group: a multiple of 16, at most this */

/*
 * Block scores: scores[(r * 4 + g) * score_stride + b] = max over tokens t of
 * block b with t < row_ctx[r] of <q_idx[r, g, :], k_t> (e4m3 codes; the index
 * key has no scale), for b < ceil(row_ctx[r] / 128); other entries are not
 * written.  q_idx: [num_rows, 4, 128] e4m3.  rows->rows_per_group (1, 2, 4 or
 * 8) consecutive rows of one request share each read of the keys.  Products
 * are exact and accumulate in fp32 on the tensor cores.  score_stride >=
 * ceil(max_ctx / 128).  A page id outside [0, num_pages) or a bad row is
 * DSA_ERR_BOUNDS on dev_status.
 */
int dsa_msa_block_scores(const void *index_pool, int64_t num_pages, const dsa_rows *rows, const uint8_t *q_idx,
                         float *scores, int64_t score_stride, int32_t *dev_status, void *stream);

/*
 * Block selection, per (row r, group g), nb = ceil(row_ctx[r] / 128): nb <= 16
 * keeps every block; otherwise block nb - 1 and the 15 highest scores among
 * blocks 0 .. nb - 2, ties to the lower block, a NaN score counting as -inf.
 * blocks[(r * 4 + g) * 16 + i] lists them ascending, -1 padded.  row_ctx
 * outside [0, max_ctx] is DSA_ERR_BOUNDS (clamped).
 */
int dsa_msa_select(const float *scores, int64_t score_stride, const int32_t *row_ctx, int32_t num_rows,
                   int32_t max_ctx, int32_t *blocks, int32_t *dev_status, void *stream);

/*
 * Block-sparse GQA attention: head h of row r belongs to group g = h / hpg
 * (hpg = heads_per_group) and attends to the visible tokens (t < row_ctx[r])
 * of its group's selected blocks:
 *   out[r, h, :] = sum_t softmax_t(sm_scale * <q_scale q[r,h,:], k_scale K_g,t>) v_scale V_g,t
 *   lse[r, h]    = natural log of the softmax denominator's sum, with the max folded in
 * q: [num_rows, 4 * hpg, 128] e4m3 codes; out: fp32 [num_rows, 4 * hpg, 128];
 * lse: fp32 [num_rows, 4 * hpg] or NULL.  A head with no visible selected
 * token gets out = 0 and lse = -inf.  S = Q K^T runs on FP8 tensor cores
 * (exact products, fp32 accumulation); P is fp16 and V is decoded exactly to
 * fp16 for P V.  The workspace (dsa_msa_attention_workspace_size bytes,
 * 256-byte aligned) holds one normalised part per selected block, merged by
 * log-sum-exp.  A selected block at or past ceil(row_ctx / 128) or a page id
 * outside the pool is DSA_ERR_BOUNDS.
 */
int dsa_msa_attention(const void *kv_pool, int64_t num_pages, float k_scale, float v_scale, const dsa_rows *rows,
                      const uint8_t *q, float q_scale, int32_t heads_per_group, const int32_t *blocks, float sm_scale,
                      float *out, float *lse, void *workspace, size_t workspace_bytes, int32_t *dev_status,
                      void *stream);

/* Workspace bytes dsa_msa_attention needs for num_rows rows. */
size_t dsa_msa_attention_workspace_size(int32_t num_rows, int32_t heads_per_group);

/*
 * ---- The dense K/V path: rotary positions, insert into a paged K/V pool, and attention of new
 * tokens over all of it.  The two sparse layers above sit next to full-attention layers, and both
 * take queries, keys and latents whose rotary dims are already rotated: these calls are that
 * chain, rope -> insert -> attention, over a K/V pool with the MSA page layout generalised:
 *
 *   page = [kv_heads] x ([K: page_size x head_dim] [V: page_size x head_dim])
 *
 * in bf16 (DSA_KV_BF16) or e4m3 codes with one fp32 scale for K and one for V (DSA_KV_FP8: value =
 * code * scale; with 4 KV heads, head_dim 128 and 128-token pages, exactly the pool
 * dsa_msa_attention reads).  page_size is 16, 32, 64 or 128, head_dim 64 or 128.  dsa_rows.
 * block_table then holds ids of these pages (bt_stride >= ceil(max_ctx / page_size)); token t of a
 * request is row t % page_size of page block_table[req][t / page_size], its slot page * page_size
 * + t % page_size.
 */
#define DSA_KV_BF16 5
#define DSA_KV_FP8 6
#define DSA_KV_MAX_HPG 128          /* query heads per KV head */
#define DSA_KV_MAX_CTX (1 << 30)    /* max_ctx of dsa_kv_attention */

typedef struct dsa_kv_cache {
    void *base;         /* device, 16-byte aligned */
    int32_t format;     /* DSA_KV_BF16 or DSA_KV_FP8 */
    int32_t page_size;  /* 16, 32, 64 or 128 tokens */
    int64_t num_pages;  /* num_pages * kv_heads * 2 * page_size < 2^31 */
    int32_t kv_heads;
    int32_t head_dim;   /* 64 or 128 */
    float k_scale;      /* DSA_KV_FP8: value of a K code = code * k_scale; ignored for DSA_KV_BF16 */
    float v_scale;
} dsa_kv_cache;

/* Element types of dsa_rope's tensors. */
#define DSA_DTYPE_BF16 1
#define DSA_DTYPE_FP32 2

/* Which elements of the rotary part form a pair: 2i and 2i + 1, or i and i + rot_dim / 2. */
#define DSA_ROPE_INTERLEAVED 0
#define DSA_ROPE_HALF 1

/* Frequencies stretched for contexts longer than the trained one (dsa_rope_frequencies). */
#define DSA_ROPE_SCALE_NONE 0
#define DSA_ROPE_SCALE_LINEAR 1
#define DSA_ROPE_SCALE_NTK 2
#define DSA_ROPE_SCALE_YARN 3

#define DSA_ROPE_MAX_DIM 256
#define DSA_ROPE_MAX_TENSORS 4

/*
 * Host-only helper: the angle per position of each of the rot_dim / 2 pairs, and the factor on the
 * rotated values, from the base theta > 1 and a context stretch `factor` >= 1 (not used by
 * DSA_ROPE_SCALE_NONE).  With f_i = theta^(-2i / rot_dim):
 *   NONE    inv_freq_i = f_i, scale 1
 *   LINEAR  f_i / factor, scale 1
 *   NTK     f_i of the base theta * factor^(rot_dim / max(rot_dim - 2, 1)), scale 1
 *   YARN    f_i (1 - r_i) + f_i / factor * r_i, scale 0.1 ln(factor) + 1; r_i rises from 0 to 1 over
 *           the pairs from the one that turns 32 times within trained_ctx positions to the one that
 *           turns once (Peng et al. 2023, "YaRN"): r_i = clamp((i - lo) / max(hi - lo, 0.001)), lo =
 *           max(floor(e(32)), 0), hi = min(ceil(e(1)), rot_dim - 1), e(n) = rot_dim ln(trained_ctx /
 *           (2 pi n)) / (2 ln theta)
 * inv_freq: host, rot_dim / 2 doubles; scale: host.
 */
int dsa_rope_frequencies(int32_t rot_dim, double theta, int32_t scaling, double factor, int32_t trained_ctx,
                         double *inv_freq, float *scale);

/*
 * Host-only helper: num_pairs angles per position (radians, finite) as the kernels take them: the
 * fraction of a turn, inv_freq / 2 pi mod 1, in units of 2^-64 turn.  A position's phase is then
 * one 64-bit product that wraps exactly, so far positions lose no precision.  inv_freq, turns: host.
 */
int dsa_rope_turns(const double *inv_freq, int32_t num_pairs, uint64_t *turns);

/* A call's angles. */
typedef struct dsa_rope_spec {
    const uint64_t *turns;    /* device [rot_dim / 2], from dsa_rope_turns */
    const int32_t *positions; /* device [num_tokens]; a negative position leaves its token out */
    int32_t rot_dim;          /* even, 2 .. DSA_ROPE_MAX_DIM */
    float scale;              /* factor on the rotated values (finite) */
} dsa_rope_spec;

/* One tensor [num_tokens, num_heads, rot_dim]: the rotary part of every head alone, in place inside
 * larger heads through its strides (in elements).  x may equal out (with equal strides); an output
 * overlaps nothing else that the call reads or writes.  What can be told from the layouts is
 * DSA_ERR_INVALID_ARG: tensors at one address, and any overlap of tensors whose tokens follow one
 * another at the same distance (parts of one packed projection) or of a single token. */
typedef struct dsa_rope_tensor {
    const void *x;
    void *out;
    int32_t num_heads;
    int32_t layout; /* DSA_ROPE_INTERLEAVED or DSA_ROPE_HALF */
    int64_t x_token_stride, x_head_stride;
    int64_t out_token_stride, out_head_stride;
} dsa_rope_tensor;

/*
 * Rotary positions of 1 .. DSA_ROPE_MAX_TENSORS tensors of the same tokens, in one launch (a
 * decode step's query heads, latent and index key).  For each pair (a, b) of token n with angle
 * t = positions[n] * inv_freq_i:
 *   out_a = scale (a cos t - b sin t),  out_b = scale (a sin t + b cos t)
 * in fp32, rounded once to dtype (of every tensor).  Elements outside the rotary part are neither
 * read nor written; a token at a negative position (padding) is not written.  tensors: host array.
 */
int dsa_rope(const dsa_rope_spec *rope, const dsa_rope_tensor *tensors, int32_t num_tensors, int32_t dtype,
             int32_t num_tokens, void *stream);

/*
 * Positions of several axes (time, height and width of images and video, say): each pair of the
 * rotary part turns with one of them, and a text token has the same position on all.
 */
#define DSA_ROPE_MAX_AXES 4
#define DSA_ROPE_AXES_SPLIT 0 /* the first sections[0] pairs are axis 0's, the next sections[1] axis 1's, ... */
#define DSA_ROPE_AXES_CYCLE 1 /* the axes in turn, pair by pair, each while it has pairs left */

/*
 * Host-only helper: the axis of each pair from the pairs that each axis has (sections: host,
 * num_axes counts >= 0 of together num_pairs) into axis (host, num_pairs bytes).
 */
int dsa_rope_sections(const int32_t *sections, int32_t num_axes, int32_t order, int32_t num_pairs, uint8_t *axis);

/* A call's angles, with several positions a token. */
typedef struct dsa_rope_axes {
    const uint64_t *turns;    /* device [rot_dim / 2], from dsa_rope_turns */
    const int32_t *positions; /* device [num_axes, num_tokens], axes axis_stride elements apart; a token
                                 with a negative position on any axis is left out */
    int64_t axis_stride;      /* >= 0; 0: one position for all axes */
    const uint8_t *axis;      /* host [rot_dim / 2]: the axis of each pair, below num_axes */
    int32_t num_axes;         /* 1 .. DSA_ROPE_MAX_AXES */
    int32_t rot_dim;          /* even, 2 .. DSA_ROPE_MAX_DIM */
    float scale;              /* factor on the rotated values (finite) */
} dsa_rope_axes;

/* dsa_rope with pair i of token n turned by positions[axis[i]][n] * inv_freq_i; everything else as there. */
int dsa_rope_with_axes(const dsa_rope_axes *rope, const dsa_rope_tensor *tensors, int32_t num_tensors, int32_t dtype,
                       int32_t num_tokens, void *stream);

/* New tokens' keys and values: [num_tokens, kv_heads, head_dim] bf16 with heads packed, tokens
 * k_stride / v_stride elements apart (parts of a packed projection output). */
typedef struct dsa_kv_rows {
    const uint16_t *k;
    const uint16_t *v;
    int64_t k_stride, v_stride;
    int32_t rot_offset; /* with a dsa_rope_spec: first rotary dim of a K head */
    int32_t layout;     /* with a dsa_rope_spec: DSA_ROPE_INTERLEAVED or DSA_ROPE_HALF */
} dsa_kv_rows;

/*
 * Write new tokens into the K/V pool: for each i with slots[i] >= 0, K and V at that slot, as
 *   DSA_KV_BF16: the values (rotated K rounded once from fp32)
 *   DSA_KV_FP8:  e4m3(x / scale), IEEE fp32 division, round to nearest even, saturating to +-448
 * rope != NULL rotates K's dims [rot_offset, rot_offset + rot_dim) on the way, in fp32, and with q
 * != NULL also rotates q (bf16, [num_tokens, q->num_heads, rot_dim]) as dsa_rope does, in the same
 * launch; q needs rope, and its output overlaps neither k, v nor the pool.  slots: device
 * [num_tokens], distinct (a slot listed twice holds bytes of either token, in any mixture).  A
 * slot outside the pool, or a slot >= 0 of a token at a negative position, is DSA_ERR_BOUNDS and
 * not written; every other byte of the pool keeps its value.
 */
int dsa_kv_insert(const dsa_kv_cache *cache, const int32_t *slots, int32_t num_tokens, const dsa_kv_rows *kv,
                  const dsa_rope_spec *rope, const dsa_rope_tensor *q, int32_t *dev_status, void *stream);

/* dsa_kv_insert with positions of several axes: K and q are rotated as dsa_rope_with_axes
 * does, and a slot >= 0 of a token with a negative position on any axis is DSA_ERR_BOUNDS. */
int dsa_kv_insert_with_axes(const dsa_kv_cache *cache, const int32_t *slots, int32_t num_tokens, const dsa_kv_rows *kv,
                            const dsa_rope_axes *rope, const dsa_rope_tensor *q, int32_t *dev_status, void *stream);

/*
 * Dense attention of new tokens over the paged cache: head h of row r reads KV head
 * g = h / (num_heads / kv_heads) and attends to the tokens t < row_ctx[r]:
 *   out[r, h, :] = sum_t softmax_t(sm_scale * <q[r,h,:], K_g,t>) V_g,t
 *   lse[r, h]    = ln sum_t exp(sm_scale * <q[r,h,:], K_g,t>)
 * q: bf16 [num_rows, num_heads, head_dim], rows q_stride elements apart (a multiple of 8), 16-byte
 * aligned; num_heads a multiple of kv_heads, at most DSA_KV_MAX_HPG times it; out: bf16 [num_rows,
 * num_heads, head_dim], 16-byte aligned; lse: fp32 [num_rows, num_heads] or NULL.  A head with no
 * visible token, or whose visible scores are all -inf, gets out = 0 and lse = -inf.  An infinity
 * of V (bf16 pool) that it sees makes its dim infinite, or NaN beside one of the other sign or
 * where its weight is 0 in fp32.  What slots at or past row_ctx[r] hold never reaches row r (NaN
 * included).  rows->rows_per_group (1, 2, 4 or 8) consecutive rows of one request (speculative
 * verify) share each read of the cache.
 *
 * Each row's tokens are split into parts by its own context (the group's largest), merged by
 * log-sum-exp, and a row's bits depend on nothing outside its group (batch invariance): the
 * workspace (device, 256-byte aligned, dsa_kv_attention_workspace_size bytes, no initial contents;
 * NULL when that is 0) holds the parts in fp32 and serves one call at a time: calls that may run
 * at once, captured graphs among them, have one each.  Outputs overlap no input (out or lse over
 * q, or over one another: DSA_ERR_INVALID_ARG).  Scores and sums are fp32.  The softmax weights
 * multiply V as the sum of two bf16 terms (bf16 pool) or rounded to fp16 (FP8 pool), where they
 * keep steps of 2^-29 of the largest of their part (head_dim 64: 2^-31) or better.  Over an FP8
 * pool q is scaled by a power of two per head and rounded to fp16 (head_dim 64) or to the sum of
 * two e4m3 terms (128: exact down to 2^-9 of the head's largest element, smaller ones within 2^-17
 * of that largest); a head of head_dim 128 with an infinity or a NaN in q gets NaN.  A row_ctx
 * outside [0, max_ctx], a row_req outside the block table or rows of a group with different
 * requests are DSA_ERR_BOUNDS, and their group gets out = 0 and lse = -inf; a page id outside the
 * pool is DSA_ERR_BOUNDS, and page 0 is read in its place.
 */
int dsa_kv_attention(const dsa_kv_cache *cache, const dsa_rows *rows, const uint16_t *q, int64_t q_stride,
                     int32_t num_heads, float sm_scale, uint16_t *out, float *lse, void *workspace,
                     size_t workspace_bytes, int32_t *dev_status, void *stream);

/* Workspace bytes dsa_kv_attention needs for num_rows rows of num_heads heads and contexts up to
 * max_ctx; 0 when every row is one part. */
size_t dsa_kv_attention_workspace_size(const dsa_kv_cache *cache, int32_t num_rows, int32_t num_heads,
                                       int32_t max_ctx);

/*
 * dsa_kv_attention of a batch whose rows share a prefix: rows first_row[s] .. first_row[s + 1] - 1 make
 * segment s, and the first shared_ctx[s] tokens of their requests are the same (their block tables list
 * the same pages there, or pages that hold the same).  Outputs are those of dsa_kv_attention, but the
 * shared tokens are read once for all rows of a segment, by the block table of the first of them that sees
 * any token: as many of them as every such row sees, in whole tiles of 128 (and none for a segment of one
 * row group, which shares its reads already); each row reads the rest by its own table.
 *
 * Rows before first_row[0] and from first_row[num_segments] on are in no segment.  first_row ascends (an
 * empty segment is allowed), from 0 at least to num_rows at most, at whole row groups; a segment that does not,
 * or with a negative shared_ctx, is DSA_ERR_BOUNDS, and its rows are as if in none.
 */
typedef struct dsa_kv_segments {
    const int32_t *first_row;  /* device [num_segments + 1] (dsa_kv_step.segment_rows) */
    const int32_t *shared_ctx; /* device [num_segments] */
    int32_t num_segments;      /* 0: plain dsa_kv_attention */
    int64_t least_saved;       /* bytes of the pool that sharing has to save in a segment, or its rows read by
                                  themselves; 0: the library's choice, by the call's shapes (num_rows and max_ctx
                                  among them: a max_ctx near the longest context leaves a call that is too small
                                  to dsa_kv_attention) and then by segment; 1: any */
} dsa_kv_segments;

/*
 * Everything not said above is as in dsa_kv_attention.  A row's bits depend on its segment and the call's shapes (and
 * on least_saved: a segment in which too little would be saved is read row by row).
 * workspace: dsa_kv_attention_shared_workspace_size bytes, otherwise as there.  Over the shared tokens of a
 * bf16 pool the softmax weights are rounded to bf16, of an FP8 pool to fp16 (in steps of 2^-31 of their
 * part's largest).
 */
int dsa_kv_attention_shared(const dsa_kv_cache *cache, const dsa_rows *rows, const dsa_kv_segments *segments,
                            const uint16_t *q, int64_t q_stride, int32_t num_heads, float sm_scale, uint16_t *out,
                            float *lse, void *workspace, size_t workspace_bytes, int32_t *dev_status, void *stream);

/* Workspace bytes of dsa_kv_attention_shared for num_rows rows in num_segments segments. */
size_t dsa_kv_attention_shared_workspace_size(const dsa_kv_cache *cache, int32_t num_rows, int32_t num_heads,
                                              int32_t max_ctx, int32_t num_segments);

/*
 * ---- A step's rows, slots and pages from the lengths of its requests (dsa_kv_plan): the row_req,
 * row_ctx, positions, slots and block table that the calls above take, made on the device, so that
 * a serving loop (or a captured graph of one) needs no host between its steps, as long as it does not
 * give up a prefix.
 *
 * Request i has context[i] tokens in the cache, listed by its row of the block table, and gets
 * new_tokens[i] >= 0 more; -1: it has ended, and its pages from first_own[i] on (those before belong
 * to a prefix that others use too) go back to the free ones.  Nobody counts a prefix's users here: its
 * pages stay taken when the last one ends, until whoever keeps that count puts them on the stack
 * between two steps.  Free pages are a stack, free_count[0]
 * entries of free_pages, the last one taken first: what ended requests give back is put on it, in
 * the order of requests and pages, then the others' new pages are taken, in that order too.  With
 *   need_i = ceil((context_i + new_i) / page_size) - ceil(context_i / page_size)
 *   wide_i = new_i raised to a multiple of rows_per_group
 * request i gets its tokens if the pages needed by requests 0 .. i are at hand and their rows fit
 * max_rows (one that needs none of the one is not held up by the other); else it gets none of them
 * and no page.
 * Rows: request after request, wide_i each (also where it gets nothing).  Row j < granted_i: row_req =
 * i, positions = context_i + j, row_ctx one more, slots = the position's slot.  Every other row, up to
 * max_rows, is padding: positions and slots -1, row_ctx 0, row_req i (behind the last request's: 0).
 * Bit for bit reproducible.  Lengths that cannot be (context < 0 or longer than a row of the table lists,
 * together with the new tokens too, new_tokens < -1, first_own < 0) are DSA_ERR_BOUNDS, and their
 * request is as one without new tokens, which gives no page back either; its context_out is its context
 * or, with new_tokens -1, 0.  So the pages of an ended request with such lengths stay taken, and its row of the
 * table, left as it was, lists them: a call in which its context and first_own are put right, and new_tokens is
 * -1 again, gives them back.  A page id outside the pool in a row's place is DSA_ERR_BOUNDS too, with slot -1;
 * so are a free_count outside [0, free_capacity] (taken as the nearer one), pages given back beyond
 * free_capacity (which are lost), and, unless `granted` is there to tell, a request that gets nothing.
 */
#define DSA_KV_PLAN_MAX_REQUESTS 16384

typedef struct dsa_kv_step {
    int32_t num_requests;          /* 0 .. DSA_KV_PLAN_MAX_REQUESTS */
    int32_t page_size;             /* 16, 32, 64 or 128 */
    int64_t num_pages;             /* of the pool; num_pages * page_size < 2^31 */
    const int32_t *context;        /* device [num_requests] */
    const int32_t *new_tokens;     /* device [num_requests] */
    const int32_t *first_own;      /* device [num_requests], or NULL: 0 */
    int32_t *block_table;          /* device [num_requests, bt_stride]; entries of new pages are written */
    int64_t bt_stride;
    int32_t *free_pages;           /* device [free_capacity]; entries given back are written */
    const int32_t *free_count;     /* device [1] */
    int32_t free_capacity;
    int32_t num_segments;          /* 0: none */
    const int32_t *segment_requests; /* device [num_segments + 1] requests, 0 .. num_requests */
    int32_t max_rows;              /* a multiple of rows_per_group */
    int32_t rows_per_group;        /* 1, 2, 4 or 8 */
    int32_t *row_req;              /* device [max_rows] */
    int32_t *row_ctx;              /* device [max_rows] */
    int32_t *positions;            /* device [max_rows], or NULL */
    int32_t *slots;                /* device [max_rows], or NULL */
    int32_t *row_start;            /* device [num_requests + 1] first row of each request and the end, or NULL */
    int32_t *granted;              /* device [num_requests] tokens that it gets, or NULL */
    int32_t *context_out;          /* device [num_requests] context + granted (0 if ended); may be context, or NULL */
    int32_t *free_count_out;       /* device [1]; may be free_count, or NULL */
    int32_t *segment_rows;         /* device [num_segments + 1] first row of each segment_requests' request */
} dsa_kv_step;

/* Outputs overlap nothing else (DSA_ERR_INVALID_ARG), except where a comment above says so. */
int dsa_kv_plan(const dsa_kv_step *step, int32_t *dev_status, void *stream);

/*
 * Failure-path self-test (no counterpart on the pages): one CTA whose
 * threads wait on a barrier that nothing ever arrives on.  The wait is the
 * bounded wait every kernel of the library uses; it gives up after the
 * library's wait limit (4e9 SM cycles, about two seconds), writes
 * DSA_ERR_TIMEOUT to dev_status (required), and every other waiter of the CTA
 * then leaves at once.  The kernel exits normally: nothing faults or hangs,
 * and the context stays usable.  Returns DSA_OK once launched.
 */
int dsa_selftest_wait_timeout(int32_t *dev_status, void *stream);

/* Human-readable text of a status code (static storage). */
const char *dsa_status_string(int status);

/* Library version, major * 10000 + minor * 100 + patch. */
int dsa_version(void);

#ifdef __cplusplus
}
#endif

#endif /* DSA_H_ */
