// kv_attention.cu -- dense attention of new tokens over the paged K/V pool (dsa_kv_attention).
//
//   out[r, h, :] = sum_t softmax_t(sm_scale <q[r,h,:], K_g,t>) V_g,t   over t < row_ctx[r]
//
// What bounds it: the cache's bytes.  A token's K and V (4 D bytes in bf16, 2 D in e4m3) serve the
// columns of one KV head, N = rows of the group x query heads per KV head, at 4 D FLOP each, so 16
// columns need 16 to 32 FLOP per byte: about 100 to 215 TFLOP/s at the HBM's rate.
//
// Split: one CTA per (row group, KV head, part of the context); the part's size goes by the group's
// context alone (kv_part), so a row's bits do not depend on its batch.  A part's (base, sum, output)
// goes to the workspace in fp32 and kv_combine_kernel merges a row's parts by log-sum-exp.
//
// In a CTA a producer warp streams 64-token tiles of K and V by TMA into a ring of stages, and four
// consumer warps share out the columns (16 each) and the tile's tokens.  Each consumer is on its own:
// it waits for a stage, takes its 16-token steps through
//     S = Q K^T      mma m16n8k16, the 16 columns on M, Q in registers for the whole part
//     P = 2^(S - b)  b a lazy base: it moves (and the output is rescaled) only when a score exceeds it
//                    by 15, so that most steps need no reduction across lanes
//     O^T += V^T P^T mma m16n8k16, 16 of the D dims on M; S's accumulator layout is this product's
//                    B operand as it stands, so P never leaves the registers
// and releases the stage; nothing synchronises the consumers until the part's end.  The contraction
// per byte is small enough that warp-level MMAs keep up with the HBM (2 cycles per SM for an m16n8k16
// measured; 64 of them per 16 tokens and 16 columns of a bf16 pool against the 356 cycles its 8 KB
// take), and they leave the running sums in registers: no TMEM round trip per tile.
//
// Precision.  bf16 pool: products are exact in fp32; a weight rounded to bf16 (2^-9) would add as much
// error as rounding the output does, so P enters as hi + lo bf16 terms (2^-17).  FP8 pool: e4m3 codes
// are exact in fp16; q is scaled by a power of two per column to fit fp16's range (exact but for
// elements 2^-25 below the column's largest), P is one fp16 term (2^-12), scaled by 2^7 so that weights
// down to 2^-21 of the base stay normal.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <atomic>
#include <type_traits>

#include "kernels.h"
#include "ptx.cuh"

namespace dsa {

namespace {

constexpr int kConsumers = 4;                     // consumer warps
constexpr int kThreads = 32 * (kConsumers + 1);   // and the producer
constexpr int kTile = 64;                         // tokens of a stage
constexpr int kStep = 16;                         // tokens of an MMA step
constexpr float kHeadroom = 15.0f;                // weights reach 2^15 (fp16 holds 65504) ...
constexpr float kBias = 7.0f;                     // ... and a moved base leaves the largest at 2^7

// The tokens of a part: as few as 128, doubled until at most max_parts cover the context.
__host__ __device__ __forceinline__ int32_t kv_part(int32_t ctx, int32_t max_parts) {
    int64_t p = 128;
    while (p * max_parts < ctx) p *= 2;
    return static_cast<int32_t>(p < ctx ? p : (ctx > 0 ? p : 128));
}

// Parts of a long context: 256 over all KV heads, so that one request alone fills the 152 SMs about
// twice, but at least 32.
__host__ __device__ __forceinline__ int32_t kv_max_parts(int32_t kv_heads) {
    return kv_heads >= 8 ? 32 : kv_heads >= 4 ? 64 : kv_heads >= 2 ? 128 : 256;
}

__host__ __device__ __forceinline__ int32_t kv_parts(int32_t ctx, int32_t max_parts) {
    const int32_t p = kv_part(ctx, max_parts);
    return ctx <= 0 ? 1 : (ctx + p - 1) / p;
}

// Bound of kv_parts over every context up to max_ctx.
int32_t kv_parts_bound(int32_t max_ctx, int32_t max_parts) {
    const int32_t n = static_cast<int32_t>((static_cast<int64_t>(max_ctx) + 127) / 128);
    return n < 1 ? 1 : (n < max_parts ? n : max_parts);
}

template <bool kFp8, int D>
struct KvCfg {
    static constexpr int kRowBytes = D * (kFp8 ? 1 : 2);
    static constexpr int kBoxBytes = kRowBytes < 128 ? kRowBytes : 128;  // a TMA box is one swizzle span wide
    static constexpr int kBoxes = kRowBytes / kBoxBytes;                 // boxes side by side in a row
    static constexpr int kPlane = kTile * kBoxBytes;                     // one box column of a tile
    static constexpr int kSide = kTile * kRowBytes;                      // K (or V) of a tile
    static constexpr int kStageBytes = 2 * kSide;
    static constexpr int kStages = 96 * 1024 / kStageBytes;  // two CTAs per SM share its 227 KB
    static constexpr int kMergeStride = D + 4;
    static constexpr int kMergeBytes = kConsumers * 16 * kMergeStride * 4;
    static_assert(kMergeBytes <= kStages * kStageBytes, "the merge reuses the stages");
    static constexpr int OFF_BARS = kStages * kStageBytes;
    static constexpr int OFF_ML = OFF_BARS + 2 * kStages * 8;
    static constexpr int OFF_MISC = OFF_ML + kConsumers * 16 * 2 * 4;
    static constexpr int kSmemBytes = OFF_MISC + 16 + 1024;  // + slack for 1024-byte alignment
};

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

__device__ __forceinline__ void ldsm4_t(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

template <bool kHalf>
__device__ __forceinline__ void mma16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if constexpr (kHalf)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                     "{%0, %1, %2, %3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                     "{%0, %1, %2, %3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Four e4m3 codes as two fp16 pairs (exact).
__device__ __forceinline__ void e4m3x4_to_f16(uint32_t v, uint32_t &lo, uint32_t &hi) {
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(v));
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}

__device__ __forceinline__ float bf16_lo(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t v) { return __uint_as_float(v & 0xffff0000u); }

// Byte offset of 16-byte unit `u` of token `t` in a side (K or V) of a stage, as its TMA boxes landed.
template <typename C>
__device__ __forceinline__ uint32_t unit_at(int t, int u) {
    if constexpr (C::kBoxBytes == 128)
        return static_cast<uint32_t>((u >> 3) * C::kPlane + t * 128 + (((u & 7) ^ (t & 7)) << 4));
    else  // 64-byte swizzle
        return static_cast<uint32_t>(t * 64 + ((u ^ ((t >> 1) & 3)) << 4));
}

// kWide: more than 8 columns per warp (two n-tiles of the second product).  kColWarps: consumer warps
// side by side over the columns; the others split the tile's tokens.
template <bool kFp8, int D, bool kWide, int kColWarps>
__global__ void __launch_bounds__(kThreads, 2)
    kv_attention_kernel(const __grid_constant__ CUtensorMap kv_map, const __grid_constant__ KvAttnArgs a) {
    using C = KvCfg<kFp8, D>;
    constexpr int kTokWarps = kConsumers / kColWarps;
    constexpr int NT = kWide ? 2 : 1;
    constexpr int KS = D / 16;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + C::OFF_BARS);
    uint64_t *empty = full + C::kStages;
    float2 *ml = reinterpret_cast<float2 *>(smem + C::OFF_ML);  // [consumer][16] base and sum
    volatile int *abort = reinterpret_cast<volatile int *>(smem + C::OFF_MISC);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        *abort = 0;
        for (int s = 0; s < C::kStages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], kConsumers);
        }
        fence_mbar_init();
        prefetch_tensormap(&kv_map);
    }
    __syncthreads();
    pdl_wait();
    pdl_launch_dependents();

    // the item: part fastest, then column block, KV head, row group
    uint32_t item = blockIdx.x;
    const int part = static_cast<int>(item % a.parts_bound);
    item /= a.parts_bound;
    const int col0 = static_cast<int>(item % a.col_blocks) * (16 * kColWarps);
    item /= a.col_blocks;
    const int g = static_cast<int>(item % a.kv_heads), row0 = static_cast<int>(item / a.kv_heads) * a.group;

    const int req = a.row_req[row0];
    int ctx = 0;       // the group's longest context
    int ctx_min = INT32_MAX;
    bool bad = req < 0 || req >= a.num_requests;
    for (int i = 0; i < a.group; ++i) {
        const int n = a.row_ctx[row0 + i];
        bad |= n < 0 || n > a.max_ctx || a.row_req[row0 + i] != req;
        ctx = max(ctx, n);
        ctx_min = min(ctx_min, n);
    }
    if (bad) {
        if (threadIdx.x == 0) report(a.status, DSA_ERR_BOUNDS);
        ctx = ctx_min = 0;
    }
    const int part_tokens = kv_part(ctx, a.max_parts), parts = kv_parts(ctx, a.max_parts);
    if (part >= parts) return;
    const int t_begin = part * part_tokens, t_end = t_begin + min(ctx - t_begin, part_tokens);
    const int tiles = (t_end - t_begin + kTile - 1) / kTile;

    float o[KS][NT][4] = {};
    float base[2] = {-INFINITY, -INFINITY}, sum[2] = {0.f, 0.f};
    const int cw = warp % kColWarps, tw = warp / kColWarps;
    const int gi = lane >> 2, ji = lane & 3;

    if (warp == kConsumers) {
        // ---- producer: boxes of min(page, tile) rows, lane b issues box b of a tile
        const int box_rows = min(a.page_size, kTile);
        const int pages_per_tile = kTile / box_rows;
        const uint64_t policy = l2_evict_first_policy();
        const int first_page = t_begin / a.page_size, num_pages = (t_end + a.page_size - 1) / a.page_size;
        const int32_t *table = a.block_table + static_cast<int64_t>(req) * a.bt_stride;
        auto load_ids = [&](int p) { return p + lane < num_pages ? table[p + lane] : 0; };
        int batch = first_page;  // page ids batch .. batch + 31 are in `ids`, one per lane
        int32_t ids = load_ids(batch), ids_next = load_ids(batch + 32);
        int issued = 0;
        for (int i = 0; i < tiles; ++i) {
            const int s = i % C::kStages;
            if (i >= C::kStages && !mbar_wait_warp(&empty[s], (i / C::kStages - 1) & 1, abort, a.status)) break;
            const int t0 = t_begin + i * kTile;
            const int boxes_here = min(pages_per_tile, (t_end - t0 + box_rows - 1) / box_rows);  // pages with tokens
            const int p0 = t0 / a.page_size;
            if (p0 >= batch + 32) {
                batch += 32;
                ids = ids_next;
                ids_next = load_ids(batch + 32);
            }
            // box b: page b / (2 kBoxes) of the tile, its K or V, its column of 128 bytes
            const int b_page = lane / (2 * C::kBoxes), b_v = lane / C::kBoxes % 2, b_x = lane % C::kBoxes;
            int32_t id = __shfl_sync(0xffffffffu, ids, (p0 + b_page - batch) & 31);
            if (lane == 0) mbar_arrive_expect_tx(&full[s], boxes_here * box_rows * 2 * C::kRowBytes);
            __syncwarp();
            if (b_page < boxes_here) {
                if (id < 0 || id >= a.num_pages) {
                    report(a.status, DSA_ERR_BOUNDS);
                    id = 0;
                }
                const int y = ((id * a.kv_heads + g) * 2 + b_v) * a.page_size + t0 % a.page_size;
                tma_load_2d_hint(smem + s * C::kStageBytes + b_v * C::kSide + b_x * C::kPlane +
                                     b_page * box_rows * C::kBoxBytes,
                                 &kv_map, &full[s], b_x * C::kBoxBytes, y, policy);
            }
            issued = i + 1;
        }
        if (*abort && lane == 0) {  // leave no copy in flight behind
            for (int i = max(0, issued - C::kStages); i < issued; ++i) {
                const long long t0 = clock64();
                while (!mbar_try_wait(&full[i % C::kStages], (i / C::kStages) & 1) && clock64() - t0 < kWaitTimeoutCycles) {
                }
            }
        }
    } else {
        // ---- consumer: columns n = col0 + 16 cw + {gi, gi + 8} as M rows
        const int hpg = a.num_heads / a.kv_heads, cols = a.group * hpg;
        uint32_t q[KS][4];
        float scale[2];  // log2 units per unit of S
        int cx[2];       // the columns' contexts
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            const int n = col0 + 16 * cw + gi + 8 * x;
            const bool real = n < cols;
            const int row = real ? n / hpg : 0;
            cx[x] = real && !bad ? a.row_ctx[row0 + row] : 0;
            scale[x] = a.s_scale;
            const uint16_t *src = a.q + (row0 + row) * a.q_stride +
                                  static_cast<int64_t>(g * hpg + (real ? n % hpg : 0)) * D;
            if constexpr (!kFp8) {
#pragma unroll
                for (int k = 0; k < KS; ++k) {
                    q[k][x] = real ? *reinterpret_cast<const uint32_t *>(src + k * 16 + ji * 2) : 0u;
                    q[k][2 + x] = real ? *reinterpret_cast<const uint32_t *>(src + k * 16 + 8 + ji * 2) : 0u;
                }
            } else {
                // K's codes come four dims to a lane (ldmatrix moves byte pairs): k slots 2j, 2j + 1
                // hold dims 4j, 4j + 1 and slots 2j + 8, 2j + 9 dims 4j + 2, 4j + 3; q likewise
                uint2 raw[KS];
                float amax = 0.f;
#pragma unroll
                for (int k = 0; k < KS; ++k) {
                    raw[k] = real ? *reinterpret_cast<const uint2 *>(src + k * 16 + ji * 4) : make_uint2(0u, 0u);
                    amax = fmaxf(amax, fmaxf(fmaxf(fabsf(bf16_lo(raw[k].x)), fabsf(bf16_hi(raw[k].x))),
                                             fmaxf(fabsf(bf16_lo(raw[k].y)), fabsf(bf16_hi(raw[k].y)))));
                }
                amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
                amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
                // 2^e brings the column's largest |q| to [2^13, 2^14); infinities stay what they are
                int e = 0;
                if (amax > 0.f && amax <= 3.4e38f) {
                    e = 140 - static_cast<int>(__float_as_uint(amax) >> 23);
                    e = max(-120, min(120, e));
                }
                const float up = __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
                scale[x] *= __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
#pragma unroll
                for (int k = 0; k < KS; ++k) {
                    q[k][x] = pack_f16(bf16_lo(raw[k].x) * up, bf16_hi(raw[k].x) * up);
                    q[k][2 + x] = pack_f16(bf16_lo(raw[k].y) * up, bf16_hi(raw[k].y) * up);
                }
            }
        }
        // the rows of the group among this warp's columns
        const int row_lo = (col0 + 16 * cw) / hpg, row_hi = min(col0 + 16 * cw + 15, cols - 1) / hpg;
        const bool idle = col0 + 16 * cw >= cols;

        for (int i = 0; i < tiles; ++i) {
            const int s = i % C::kStages;
            if (!mbar_wait_warp(&full[s], (i / C::kStages) & 1, abort, a.status)) break;
            const uint32_t ks = smem_u32(smem + s * C::kStageBytes), vs = ks + C::kSide;
#pragma unroll 1
            for (int st = tw; st < kTile / kStep && !idle; st += kTokWarps) {
                const int ts = st * kStep, t0 = t_begin + i * kTile + ts;  // the step's tokens, in tile and context
                if (t0 >= t_end) break;
                // S: columns gi, gi + 8; tokens t0 + 8 n + 2 ji + {0, 1}
                float c[2][4] = {};
                if constexpr (!kFp8) {
                    // matrices: tokens 0-7 (k 0-7, 8-15), tokens 8-15 (k 0-7, 8-15)
                    const int t = ts + (lane & 7) + ((lane >> 4) << 3), u = (lane >> 3) & 1;
#pragma unroll
                    for (int k = 0; k < KS; ++k) {
                        uint32_t b[4];
                        ldsm4(b, ks + unit_at<C>(t, 2 * k + u));
                        mma16<false>(c[0], q[k], b[0], b[1]);
                        mma16<false>(c[1], q[k], b[2], b[3]);
                    }
                } else {
                    const int t = ts + (lane & 7) + ((lane >> 4) << 3), u = (lane >> 3) & 1;
#pragma unroll
                    for (int k = 0; k < KS; k += 2) {
                        uint32_t b[4];
                        ldsm4(b, ks + unit_at<C>(t, k + u));
#pragma unroll
                        for (int n = 0; n < 2; ++n) {
                            uint32_t b0, b1;
                            e4m3x4_to_f16(b[2 * n], b0, b1);
                            mma16<true>(c[n], q[k], b0, b1);
                            e4m3x4_to_f16(b[2 * n + 1], b0, b1);
                            mma16<true>(c[n], q[k + 1], b0, b1);
                        }
                    }
                }
                const bool edge = t0 + kStep > ctx_min;  // some column does not see all of the step
#pragma unroll
                for (int n = 0; n < 2; ++n)
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        c[n][x] *= scale[x >> 1];
                        if (edge && t0 + 8 * n + 2 * ji + (x & 1) >= cx[x >> 1]) c[n][x] = -INFINITY;
                    }
                float top[2];
#pragma unroll
                for (int x = 0; x < 2; ++x)
                    top[x] = fmaxf(fmaxf(c[0][2 * x], c[0][2 * x + 1]), fmaxf(c[1][2 * x], c[1][2 * x + 1]));
                if (__any_sync(0xffffffffu, top[0] > base[0] + kHeadroom || top[1] > base[1] + kHeadroom)) {
                    float f[2];
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        top[x] = fmaxf(top[x], __shfl_xor_sync(0xffffffffu, top[x], 1));
                        top[x] = fmaxf(top[x], __shfl_xor_sync(0xffffffffu, top[x], 2));
                        f[x] = 1.f;  // a column whose own scores fit keeps its base
                        if (top[x] > base[x] + kHeadroom) {
                            f[x] = ex2(base[x] - (top[x] - kBias));
                            base[x] = top[x] - kBias;
                        }
                        sum[x] *= f[x];
                    }
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        const float f0 = __shfl_sync(0xffffffffu, f[n], 8 * ji), f1 = __shfl_sync(0xffffffffu, f[n], 8 * ji + 4);
#pragma unroll
                        for (int m = 0; m < KS; ++m) {
                            o[m][n][0] *= f0;
                            o[m][n][1] *= f1;
                            o[m][n][2] *= f0;
                            o[m][n][3] *= f1;
                        }
                    }
                }
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const float b = base[x] == -INFINITY ? 0.f : base[x];
#pragma unroll
                    for (int n = 0; n < 2; ++n)
#pragma unroll
                        for (int y = 0; y < 2; ++y) {
                            c[n][2 * x + y] = ex2(c[n][2 * x + y] - b);
                            sum[x] += c[n][2 * x + y];
                        }
                }
                // P^T as the second product's B operand: n-tile x holds columns 8 x + gi
                uint32_t hi[NT][2], lo[NT][2];
#pragma unroll
                for (int x = 0; x < NT; ++x)
#pragma unroll
                    for (int n = 0; n < 2; ++n) {
                        const float p0 = c[n][2 * x], p1 = c[n][2 * x + 1];
                        if constexpr (kFp8) {
                            hi[x][n] = pack_f16(p0, p1);
                        } else {
                            hi[x][n] = pack_bf16(p0, p1);
                            lo[x][n] = pack_bf16(p0 - bf16_lo(hi[x][n]), p1 - bf16_hi(hi[x][n]));
                        }
                    }
                // O^T += V^T P^T.  In an edge step the rows of the group take turns, with V's tokens at and past
                // the row's context zeroed and the other rows' columns put back: what a row does not see
                // may be NaN, and 0 x NaN must not reach its sums.
                auto product = [&](auto edge_step, int row) {
                    constexpr bool kEdge = decltype(edge_step)::value;
                    uint32_t keep[2];      // tokens 2 ji, 2 ji + 1 of either half
                    bool mine[NT][2];      // columns 8 x + 2 ji + {0, 1} are this row's
                    if constexpr (kEdge) {
                        const int n = bad ? 0 : a.row_ctx[row0 + row];
#pragma unroll
                        for (int y = 0; y < 2; ++y) {
                            const int t = t0 + 8 * y + 2 * ji;
                            keep[y] = (t < n ? 0xffffu : 0u) | (t + 1 < n ? 0xffff0000u : 0u);
                        }
#pragma unroll
                        for (int x = 0; x < NT; ++x)
#pragma unroll
                            for (int y = 0; y < 2; ++y) mine[x][y] = (col0 + 16 * cw + 8 * x + 2 * ji + y) / hpg == row;
                    }
                    auto accumulate = [&](float(&acc)[NT][4], uint32_t(&v)[4]) {
                        if constexpr (kEdge) {
#pragma unroll
                            for (int y = 0; y < 4; ++y) v[y] &= keep[y >> 1];
                        }
#pragma unroll
                        for (int x = 0; x < NT; ++x) {
                            float old[4];
#pragma unroll
                            for (int y = 0; y < 4; ++y) old[y] = acc[x][y];
                            mma16<kFp8>(acc[x], v, hi[x][0], hi[x][1]);
                            if constexpr (!kFp8) mma16<false>(acc[x], v, lo[x][0], lo[x][1]);
                            if constexpr (kEdge) {
#pragma unroll
                                for (int y = 0; y < 4; ++y) acc[x][y] = mine[x][y & 1] ? acc[x][y] : old[y];
                            }
                        }
                    };
                    if constexpr (!kFp8) {
                        // matrices: tokens 0-7 (d 0-7, 8-15), tokens 8-15 (d 0-7, 8-15)
                        const int t = ts + (lane & 7) + ((lane >> 4) << 3), u = (lane >> 3) & 1;
#pragma unroll
                        for (int m = 0; m < KS; ++m) {
                            uint32_t v[4];
                            ldsm4_t(v, vs + unit_at<C>(t, 2 * m + u));
                            accumulate(o[m], v);
                        }
                    } else {
                        // matrices: unit m tokens 0-7, 8-15, unit m + 1 likewise; a lane gets codes
                        // [t d][t d+1][t+1 d][t+1 d+1] with d = 2 gi: M row gi is dim 2 gi, row gi + 8 dim 2 gi + 1
                        const int t = ts + (lane & 15), u = lane >> 4;
#pragma unroll
                        for (int m = 0; m < KS; m += 2) {
                            uint32_t w[4];
                            ldsm4_t(w, vs + unit_at<C>(t, m + u));
#pragma unroll
                            for (int y = 0; y < 2; ++y) {
                                uint32_t v[4];
                                e4m3x4_to_f16(__byte_perm(w[2 * y], 0, 0x3120), v[0], v[1]);
                                e4m3x4_to_f16(__byte_perm(w[2 * y + 1], 0, 0x3120), v[2], v[3]);
                                accumulate(o[m + y], v);
                            }
                        }
                    }
                };
                if (!edge) {
                    product(std::false_type{}, 0);
                } else {
#pragma unroll 1
                    for (int row = row_lo; row <= row_hi; ++row) product(std::true_type{}, row);
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&empty[s]);
        }
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            sum[x] += __shfl_xor_sync(0xffffffffu, sum[x], 1);
            sum[x] += __shfl_xor_sync(0xffffffffu, sum[x], 2);
            if (ji == 0) ml[warp * 16 + gi + 8 * x] = make_float2(base[x], sum[x]);
        }
    }
    __syncthreads();  // every stage is consumed: the merge reuses them
    if (*abort) return;

    // ---- merge the token warps of each column, each in its own base
    float *merge = reinterpret_cast<float *>(smem);  // [consumer][16][kMergeStride]
    if (warp < kConsumers) {
        float f[2];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            float top = -INFINITY;
            for (int w = 0; w < kTokWarps; ++w) top = fmaxf(top, ml[(w * kColWarps + cw) * 16 + gi + 8 * x].x);
            f[x] = ex2(base[x] - (top == -INFINITY ? 0.f : top));
        }
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const float f0 = __shfl_sync(0xffffffffu, f[n], 8 * ji), f1 = __shfl_sync(0xffffffffu, f[n], 8 * ji + 4);
            float *dst = merge + (warp * 16 + 8 * n + 2 * ji) * C::kMergeStride;
#pragma unroll
            for (int m = 0; m < KS; ++m) {
                const int d0 = kFp8 ? 16 * m + 2 * gi : 16 * m + gi, d1 = kFp8 ? d0 + 1 : d0 + 8;
                dst[d0] = o[m][n][0] * f0;
                dst[C::kMergeStride + d0] = o[m][n][1] * f1;
                dst[d1] = o[m][n][2] * f0;
                dst[C::kMergeStride + d1] = o[m][n][3] * f1;
            }
        }
    }
    __syncthreads();
    const int hpg = a.num_heads / a.kv_heads, cols = min(16 * kColWarps, a.group * hpg - col0);
    for (int i = threadIdx.x; i < cols * (D / 4); i += kThreads) {
        const int n = i / (D / 4), d = i % (D / 4) * 4;
        const int w0 = n / 16, c = n % 16;
        float top = -INFINITY;
        for (int w = 0; w < kTokWarps; ++w) top = fmaxf(top, ml[(w * kColWarps + w0) * 16 + c].x);
        const float b = top == -INFINITY ? 0.f : top;
        float total = 0.f;
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int w = 0; w < kTokWarps; ++w) {
            const int at = (w * kColWarps + w0) * 16 + c;
            total += ml[at].y * ex2(ml[at].x - b);
            const float4 y = *reinterpret_cast<const float4 *>(merge + at * C::kMergeStride + d);
            x.x += y.x;
            x.y += y.y;
            x.z += y.z;
            x.w += y.w;
        }
        const int row = row0 + (col0 + n) / hpg, head = g * hpg + (col0 + n) % hpg;
        const int64_t at = static_cast<int64_t>(row) * a.num_heads + head;
        if (parts > 1) {
            *reinterpret_cast<float4 *>(a.part_o + (at * a.parts_bound + part) * D + d) = x;
            if (d == 0) a.part_ml[at * a.parts_bound + part] = make_float2(top, total);
        } else {
            const float inv = total == 0.f ? 0.f : a.v_scale / total;
            const bool none = total == 0.f;
            *reinterpret_cast<uint2 *>(a.out + at * D + d) =
                none ? make_uint2(0u, 0u) : make_uint2(pack_bf16(x.x * inv, x.y * inv), pack_bf16(x.z * inv, x.w * inv));
            if (d == 0 && a.lse != nullptr) a.lse[at] = none ? -INFINITY : (b + log2f(total)) * 0.6931471805599453f;
        }
    }
}

// Merge of a row's parts: one CTA per (row, head), one thread per dim.
template <int D>
__global__ void __launch_bounds__(D) kv_combine_kernel(const __grid_constant__ KvAttnArgs a) {
    pdl_wait();
    pdl_launch_dependents();
    const int64_t at = blockIdx.x;
    const int row0 = static_cast<int>(at / a.num_heads) / a.group * a.group;
    int ctx = 0;
    for (int i = 0; i < a.group; ++i) ctx = max(ctx, min(a.row_ctx[row0 + i], a.max_ctx));
    const int parts = kv_parts(ctx, a.max_parts);
    if (parts == 1) return;  // written by the attention kernel
    const float2 *ml = a.part_ml + at * a.parts_bound;
    const float *po = a.part_o + at * a.parts_bound * D + threadIdx.x;
    float top = -INFINITY;
    for (int p = 0; p < parts; ++p) top = fmaxf(top, ml[p].x);
    const float b = top == -INFINITY ? 0.f : top;
    float total = 0.f, x = 0.f;
#pragma unroll 8
    for (int p = 0; p < parts; ++p) {
        const float f = ex2(ml[p].x - b);
        total += ml[p].y * f;
        x += po[static_cast<int64_t>(p) * D] * f;
    }
    const bool none = total == 0.f;
    a.out[at * D + threadIdx.x] = __bfloat16_as_ushort(__float2bfloat16_rn(none ? 0.f : x * (a.v_scale / total)));
    if (threadIdx.x == 0 && a.lse != nullptr) a.lse[at] = none ? -INFINITY : (b + log2f(total)) * 0.6931471805599453f;
}

template <bool kFp8, int D, bool kWide, int kColWarps>
cudaError_t launch_variant(const CUtensorMap &map, const KvAttnArgs &a, unsigned grid, cudaStream_t s) {
    using C = KvCfg<kFp8, D>;
    auto kern = kv_attention_kernel<kFp8, D, kWide, kColWarps>;
    static std::atomic<uint64_t> configured{0};  // devices whose shared-memory limit is raised, a bit each
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = 1ull << (dev & 63);
    if (dev >= 64 || !(configured.load() & bit)) {
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmemBytes);
        if (e != cudaSuccess) return e;
        if (dev < 64) configured.fetch_or(bit);
    }
    return launch_pdl(kern, dim3(grid), dim3(kThreads), C::kSmemBytes, s, map, a);
}

template <bool kFp8, int D>
cudaError_t launch_format(const CUtensorMap &map, KvAttnArgs &a, cudaStream_t s) {
    const int cols = a.group * (a.num_heads / a.kv_heads);
    const int col_warps = cols <= 16 ? 1 : cols <= 32 ? 2 : 4;
    a.col_blocks = (cols + 16 * col_warps - 1) / (16 * col_warps);
    const int64_t grid = static_cast<int64_t>(a.num_rows / a.group) * a.kv_heads * a.col_blocks * a.parts_bound;
    if (grid > 0x7fffffff) return cudaErrorInvalidConfiguration;
    const unsigned n = static_cast<unsigned>(grid);
    if (cols <= 8) return launch_variant<kFp8, D, false, 1>(map, a, n, s);
    if (col_warps == 1) return launch_variant<kFp8, D, true, 1>(map, a, n, s);
    if (col_warps == 2) return launch_variant<kFp8, D, true, 2>(map, a, n, s);
    return launch_variant<kFp8, D, true, 4>(map, a, n, s);
}

}  // namespace

int kv_box_rows(int32_t page_size) { return page_size < kTile ? page_size : kTile; }

size_t kv_attention_workspace_bytes(int64_t num_rows, int32_t num_heads, int32_t kv_heads, int32_t head_dim,
                                    int32_t max_ctx) {
    const size_t parts = static_cast<size_t>(kv_parts_bound(max_ctx, kv_max_parts(kv_heads)));
    if (parts <= 1) return 0;
    const size_t n = static_cast<size_t>(num_rows) * static_cast<size_t>(num_heads) * parts;
    return align256(n * static_cast<size_t>(head_dim) * 4) + align256(n * 8);
}

cudaError_t launch_kv_attention(const CUtensorMap &kv_map, KvAttnArgs &a, void *workspace, cudaStream_t s) {
    if (a.num_rows == 0) return cudaSuccess;
    a.max_parts = kv_max_parts(a.kv_heads);
    a.parts_bound = kv_parts_bound(a.max_ctx, a.max_parts);
    const size_t n = static_cast<size_t>(a.num_rows) * static_cast<size_t>(a.num_heads) * a.parts_bound;
    a.part_o = static_cast<float *>(workspace);
    a.part_ml = reinterpret_cast<float2 *>(static_cast<uint8_t *>(workspace) +
                                           align256(n * static_cast<size_t>(a.head_dim) * 4));
    cudaError_t e;
    if (a.fp8) e = a.head_dim == 64 ? launch_format<true, 64>(kv_map, a, s) : launch_format<true, 128>(kv_map, a, s);
    else e = a.head_dim == 64 ? launch_format<false, 64>(kv_map, a, s) : launch_format<false, 128>(kv_map, a, s);
    if (e != cudaSuccess || a.parts_bound == 1) return e;
    const int64_t grid = static_cast<int64_t>(a.num_rows) * a.num_heads;
    if (grid > 0x7fffffff) return cudaErrorInvalidConfiguration;
    const dim3 gr(static_cast<unsigned>(grid)), b(static_cast<unsigned>(a.head_dim));
    return a.head_dim == 64 ? launch_pdl(kv_combine_kernel<64>, gr, b, 0, s, a)
                            : launch_pdl(kv_combine_kernel<128>, gr, b, 0, s, a);
}

}  // namespace dsa
