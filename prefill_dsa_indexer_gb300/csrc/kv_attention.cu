// kv_attention.cu -- dense attention of new tokens over the paged K/V pool (dsa_kv_attention).
//
//   out[r, h, :] = sum_t softmax_t(sm_scale <q[r,h,:], K_g,t>) V_g,t   over t < row_ctx[r]
//
// What bounds it: the cache's bytes.  A token's K and V (4 D bytes in bf16, 2 D in e4m3) serve the
// columns of one KV head, N = rows of the group x query heads per KV head, at 4 D FLOP each, so 16
// columns need 16 to 32 FLOP per byte: about 100 to 215 TFLOP/s at the HBM's rate.
//
// Split: an item is a (row group, KV head, part of the context); the part's size goes by the group's
// context alone (kv_parts_shift), so a row's bits do not depend on its batch.  A part's (base, sum, output)
// goes to the workspace in fp32 and kv_combine_kernel merges a row's parts by log-sum-exp.  Two
// persistent CTAs per SM take equal shares of the items, and one item's K and V stream in while the one
// before it is merged and written.  8 x 128K tokens of a bf16 pool (4 KV heads of 128, 8 query heads each):
// 317 us, the copy bandwidth; 24 x 8K 67 us against 60; 23 ragged rows of up to 9,001 tokens (3 heads of 64, 16-token
// pages): 20 us against 12 us of bytes, the rest start-up, the first tiles' latency and the merge.  FP8 of head_dim 64 (4
// KV heads, 16 query heads each): 32 x 16K-64K 112 us against 102, but 24 x 8K 34 us against 15 and 4 x 4 rows of 64K 78
// us against 20, where the codes' conversions to fp16 take the issue slots.
//
// In a CTA a producer warp streams tiles of K and V by TMA into a ring of stages, a query warp brings
// each item's queries as MMA fragments, and four consumer warps share out the columns (16 each) and
// the tile's tokens.  Each consumer is on its own: it waits for a stage, takes its 16- or 32-token
// steps through
//     S = Q K^T      the 16 columns on M, Q in registers for the whole item
//     P = 2^(S - b)  b a lazy base: it moves (and the output is rescaled) only when a score exceeds it
//                    by 15, so that most steps need no reduction across lanes
//     O^T += V^T P^T mma m16n8k16, 16 of the D dims on M; S's accumulator layout is this product's
//                    B operand as it stands, so P never leaves the registers
// and releases the stage.  The contraction per byte is small enough that warp-level MMAs keep up with
// the HBM (2 cycles per SM for an m16n8k16 measured; the 48 of them per 16
// tokens and 16 columns of a bf16 pool against the 356 cycles its 8 KB take), and they leave the
// running sums in registers: no TMEM round trip per tile.
//
// Precision.  bf16 pool: products are exact in fp32; a weight rounded to bf16 (2^-9) would add as much
// error as rounding the output does, so P enters as hi + lo bf16 terms (2^-16).  FP8 pool: e4m3 codes
// are exact in fp16; q is scaled by a power of two per column to fit fp16's range (exact but for
// elements 2^-25 below the column's largest), P is one fp16 term (2^-12), scaled by 2^7 so that weights
// down to 2^-21 of the base stay normal.  (mma.sync on e4m3 operands was tried for S: the warps spend their time in
// branches and instruction fetches there, 178 us against 108 us for 16 x 16K.)
#include <type_traits>

#include "kv_attention_common.cuh"

namespace dsa {

namespace {

using namespace kv;

constexpr int kConsumers = 4;                    // consumer warps
constexpr int kProducer = 4, kQuery = 5;         // the warp that streams K and V, the one that brings queries
constexpr int kThreads = 32 * (kConsumers + 2);
constexpr float kHeadroom = 15.0f;                // weights reach 2^15 (fp16 holds 65504) ...
constexpr float kBias = 7.0f;                     // ... and a moved base leaves the largest at 2^7

// Bound of kv_parts over every context up to max_ctx.
uint32_t kv_parts_bound(int32_t max_ctx, int32_t parts_shift) {
    const int64_t n = (static_cast<int64_t>(max_ctx) + (1 << kPartMin) - 1) >> kPartMin, most = 1ll << parts_shift;
    return static_cast<uint32_t>(n < 1 ? 1 : (n < most ? n : most));
}

// kColWarps consumer warps side by side over the columns (16 each), kTokWarps over a tile's tokens.
template <bool kFp8, int D, int kColWarps>
struct KvCfg {
    static constexpr int kTokWarps = kConsumers / kColWarps;
    static constexpr int kRowBytes = D * (kFp8 ? 1 : 2);
    static constexpr int kBoxBytes = kRowBytes < 128 ? kRowBytes : 128;  // a TMA box is one swizzle span wide
    static constexpr int kBoxes = kRowBytes / kBoxBytes;                 // boxes side by side in a row
    static constexpr int kStageBytes = kTokWarps > 1 ? 32768 : 16384;
    static constexpr int kTile = kStageBytes / (2 * kRowBytes);          // tokens of a stage
    static constexpr int kPlane = kTile * kBoxBytes;                     // one box column of a tile
    static constexpr int kSide = kTile * kRowBytes;                      // K (or V) of a tile
    static constexpr int kStages = kTokWarps > 1 ? 3 : 5;
    static constexpr int kWarpTokens = kTile / kTokWarps;                // a warp's share of a tile
    static constexpr int kSub = kWarpTokens >= 32 ? 2 : 1;               // 16-token MMA steps taken together
    static constexpr int kStepTokens = 16 * kSub;
    static constexpr int kQBytes = 16 * D * 2;                           // a column warp's queries, 16 bits each
    static constexpr int kMergeFloats = 16 * D;                          // a consumer's output
    static_assert(kTokWarps == 1 || kConsumers * kMergeFloats * 4 <= kStageBytes, "the merge fits a stage");
    static constexpr int OFF_Q = kStages * kStageBytes;
    static constexpr int OFF_COLS = OFF_Q + kColWarps * kQBytes;         // [16 kColWarps] scale and context
    static constexpr int OFF_ML = OFF_COLS + 16 * kColWarps * 8;         // [item parity][consumer][16] base and sum
    static constexpr int OFF_ITEM = OFF_ML + 2 * kConsumers * 16 * 8;
    static constexpr int OFF_SCHED = OFF_ITEM + 64;
    static constexpr int OFF_BARS = OFF_SCHED + static_cast<int>(sizeof(KvSchedule));
    static constexpr int kNumBars = 2 * kStages + 3;
    static constexpr int OFF_MISC = OFF_BARS + kNumBars * 8;
    static constexpr int kSmemBytes = OFF_MISC + 16 + 1024;              // + slack for 1024-byte alignment
    static_assert(kWarpTokens % kStepTokens == 0, "whole steps");
    static_assert(kSmemBytes <= 115712, "two CTAs per SM");
};

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
__device__ __forceinline__ void mma16(float (&c)[4], const uint4 &a, uint32_t b0, uint32_t b1) {
    if constexpr (kHalf)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                     "{%0, %1, %2, %3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                     "{%0, %1, %2, %3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1));
}

// Four e4m3 codes as two fp16 pairs (exact).
__device__ __forceinline__ void e4m3x4_to_f16(uint32_t v, uint32_t &lo, uint32_t &hi) {
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(v));
}

// Two weights as hi + lo bf16 terms.  hi is cut off, not rounded, so that lo is positive, and lo is never 0 beside a hi
// that is not: an infinity of V times the one and the other is the same infinity.
__device__ __forceinline__ void split_weights(float p0, float p1, uint32_t &hi, uint32_t &lo) {
    hi = __byte_perm(__float_as_uint(p0), __float_as_uint(p1), 0x7632);
    const uint32_t least = 0x00800080u;  // 2^-126
    const __nv_bfloat162 rest = __floats2bfloat162_rn(p0 - bf16_lo(hi), p1 - bf16_hi(hi));
    const __nv_bfloat162 some = __hmin2(*reinterpret_cast<const __nv_bfloat162 *>(&hi),
                                        *reinterpret_cast<const __nv_bfloat162 *>(&least));
    const __nv_bfloat162 l = __hmax2(rest, some);
    lo = *reinterpret_cast<const uint32_t *>(&l);
}

// Byte offset of 16-byte unit `u` of token `t` in a side (K or V) of a stage, as its TMA boxes landed.
template <typename C>
__device__ __forceinline__ uint32_t unit_at(int t, int u) {
    if constexpr (C::kBoxBytes == 128)
        return static_cast<uint32_t>((u >> 3) * C::kPlane + t * 128 + (((u & 7) ^ (t & 7)) << 4));
    else  // 64-byte swizzle
        return static_cast<uint32_t>(t * 64 + ((u ^ ((t >> 1) & 3)) << 4));
}

// Byte offset of 16-byte unit `u` of column `n` of a column warp's queries: rows of 2 D bytes, units
// swizzled so that ldmatrix's eight rows lie in different banks.
template <int D>
__device__ __forceinline__ uint32_t q_unit_at(int n, int u) {
    return static_cast<uint32_t>(n * 2 * D + ((u ^ (n & 7)) << 4));
}

// Float offset of dim `d` of column `n` in a consumer's part of the merge stage; the turned bits keep the
// MMA fragments' stores and the rows' loads free of bank conflicts.
template <int D>
__device__ __forceinline__ int merge_at(int n, int d) {
    return n * D + (d ^ ((n >> 1 & 3) << 3));
}

// The row of its group that a column belongs to.
__device__ __forceinline__ int row_of(const KvAttnArgs &a, int col) {
    return static_cast<int>(static_cast<uint32_t>(col) * a.hpg_mul >> 20);
}

// A turn of the queries: of 32 / kUnits neighbouring columns from `n` (of the CTA's) on, a unit of 16 dims per lane.
template <int D>
struct QueryTurn {
    static constexpr int kUnits = D / 16, kTurnCols = 32 / kUnits;
    uint4 v0, v1;

    __device__ __forceinline__ void load(const KvAttnArgs &a, const KvCursor &w, int n, int cols, int hpg, int lane) {
        const int col = w.col0 + n + lane / kUnits;
        v0 = v1 = make_uint4(0u, 0u, 0u, 0u);
        if (col < cols) {
            const int row = row_of(a, col);
            const uint4 *src = reinterpret_cast<const uint4 *>(a.q + (w.row0 + row) * a.q_stride +
                                                               static_cast<int64_t>(w.g * hpg + col - row * hpg) * D +
                                                               lane % kUnits * 16);
            v0 = src[0];
            v1 = src[1];
        }
    }

    // Into a column warp's place in 16 bits, columns as rows, with each column's scale and context.
    template <bool kFp8>
    __device__ __forceinline__ void put(uint8_t *queries, float2 *cols_s, const KvAttnArgs &a, const KvCursor &w, int n,
                                        int cols, int hpg, int lane) {
        const int unit = lane % kUnits;
        n += lane / kUnits;
        const int col = w.col0 + n;
        const int ctx = __shfl_sync(0xffffffffu, w.my_ctx, col < cols ? row_of(a, col) : 0);
        float scale = a.s_scale;
        if constexpr (kFp8) {
            const uint32_t h[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
            float amax = 0.f;
#pragma unroll
            for (int y = 0; y < 8; ++y) amax = fmaxf(amax, fmaxf(fabsf(bf16_lo(h[y])), fabsf(bf16_hi(h[y]))));
#pragma unroll
            for (int y = 1; y < kUnits; y <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, y));
            // 2^e brings the column's largest |q| to [2^13, 2^14); infinities and NaN stay what they are
            int e = 0;
            if (amax > 0.f && amax <= 3.4e38f) {
                e = 140 - static_cast<int>(__float_as_uint(amax) >> 23);
                e = max(-120, min(120, e));
            }
            const float up = __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
            scale *= __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
            uint32_t f[8];
#pragma unroll
            for (int y = 0; y < 8; ++y) f[y] = pack_f16(bf16_lo(h[y]) * up, bf16_hi(h[y]) * up);
            // K's codes come four dims to a lane (ldmatrix moves byte pairs): the k slots of its low
            // and high pairs hold dims 4j, 4j + 1 and 4j + 2, 4j + 3; q's in the same order
            v0 = make_uint4(f[0], f[2], f[4], f[6]);
            v1 = make_uint4(f[1], f[3], f[5], f[7]);
        }
        // a masked score is -inf times this: neither zero nor infinity
        if (unit == 0)
            cols_s[n] = make_float2(fminf(fmaxf(scale, 1.17549435e-38f), 3.40282347e38f),
                                    __int_as_float(col < cols ? ctx : 0));
        uint8_t *dst = queries + (n >> 4) * (16 * D * 2);
        *reinterpret_cast<uint4 *>(dst + q_unit_at<D>(n & 15, 2 * unit)) = v0;
        *reinterpret_cast<uint4 *>(dst + q_unit_at<D>(n & 15, 2 * unit + 1)) = v1;
    }
};

// kWide: more than 8 columns per warp (two n-tiles of the second product).
template <bool kFp8, int D, bool kWide, int kColWarps>
__global__ void __launch_bounds__(kThreads, 2)
    kv_attention_kernel(const __grid_constant__ CUtensorMap kv_map, const __grid_constant__ KvAttnArgs a) {
    using C = KvCfg<kFp8, D, kColWarps>;
    constexpr int kTokWarps = C::kTokWarps, kCols = 16 * kColWarps;
    constexpr int NT = kWide ? 2 : 1;
    constexpr int KS = D / 16, SUB = C::kSub;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + C::OFF_BARS);  // [kStages] tile landed
    uint64_t *empty = full + C::kStages;                                // [kStages] consumers are done with it
    uint64_t *q_full = empty + C::kStages, *q_empty = q_full + 1;       // an item and its queries
    uint64_t *merge = q_empty + 1;                                      // every consumer's output is in the merge stage
    float2 *cols_s = reinterpret_cast<float2 *>(smem + C::OFF_COLS);    // scale, context (int bits)
    float2 *ml_s = reinterpret_cast<float2 *>(smem + C::OFF_ML);
    KvItem *item_s = reinterpret_cast<KvItem *>(smem + C::OFF_ITEM);
    volatile int *abort = reinterpret_cast<volatile int *>(smem + C::OFF_MISC);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        *abort = 0;
        for (int s = 0; s < C::kStages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], kConsumers);
        }
        mbar_init(q_full, 1);
        mbar_init(q_empty, kConsumers);
        mbar_init(merge, kConsumers);
        fence_mbar_init();
        prefetch_tensormap(&kv_map);
    }
    __syncthreads();
    pdl_wait();
    const bool direct = kv_direct(a);
    if (direct) pdl_launch_dependents();
    KvSchedule *sched = reinterpret_cast<KvSchedule *>(smem + C::OFF_SCHED);
    kv_fill_schedule(a, sched);
    __syncthreads();

    const int hpg = a.hpg, cols = a.group * hpg;
    const int gi = lane >> 2, ji = lane & 3;
    KvCursor w;
    bool more = w.first<kCols>(a, sched, lane);
    using Turn = QueryTurn<D>;

    if (warp == kProducer) {
        // ---- K and V: boxes of at most kTile rows, lane b issues box b of a tile
        const int box_rows = min(a.page_size, C::kTile);
        const int box_shift = min(a.page_shift, 31 - __clz(C::kTile)), boxes = C::kTile >> box_shift;
        // box of this lane: token box b_t of the tile, K or V, column of 128 bytes
        const int b_t = lane / (2 * C::kBoxes), b_v = lane / C::kBoxes % 2, b_x = lane % C::kBoxes;
        const uint64_t policy = l2_evict_first_policy();
        int s = 0, issued = 0;
        uint32_t phase = 1;
        bool go = true;
        for (; more && go; more = w.next<kCols>(a, lane)) {
            const int num_pages = (w.t_end + a.page_size - 1) >> a.page_shift;
            const int32_t *table = a.block_table + static_cast<int64_t>(w.req) * a.bt_stride;
            auto load_ids = [&](int p) { return p + lane < num_pages ? table[p + lane] : 0; };
            int batch = w.t_begin >> a.page_shift;  // page ids batch .. batch + 31 are in `ids`, one per lane
            int32_t ids = load_ids(batch), ids_next = load_ids(batch + 32);
            for (int t0 = w.t_begin; t0 < w.t_end; t0 += C::kTile) {
                if (!wait_mbar_warp(&empty[s], phase, abort)) {
                    gave_up(abort, a.status);
                    go = false;
                    break;
                }
                const int here = min(boxes, (w.t_end - t0 + box_rows - 1) >> box_shift);  // boxes with tokens
                if ((t0 >> a.page_shift) >= batch + 32) {
                    batch += 32;
                    ids = ids_next;
                    ids_next = load_ids(batch + 32);
                }
                const int tb = t0 + b_t * box_rows;
                int32_t id = __shfl_sync(0xffffffffu, ids, ((tb >> a.page_shift) - batch) & 31);
                if (lane == 0) mbar_arrive_expect_tx(&full[s], here * box_rows * 2 * C::kRowBytes);
                __syncwarp();
                if (b_t < here) {
                    if (id < 0 || id >= a.num_pages) {
                        report(a.status, DSA_ERR_BOUNDS);
                        id = 0;
                    }
                    const int y = ((id * a.kv_heads + w.g) * 2 + b_v) * a.page_size + (tb & (a.page_size - 1));
                    tma_load_2d_hint(smem + s * C::kStageBytes + b_v * C::kSide + b_x * C::kPlane +
                                         b_t * box_rows * C::kBoxBytes,
                                     &kv_map, &full[s], b_x * C::kBoxBytes, y, policy);
                }
                ++issued;
                if (++s == C::kStages) {
                    s = 0;
                    phase ^= 1;
                }
            }
            if (kTokWarps > 1 && go) {  // the next stage is the consumers', to merge the item's output in
                if (!wait_mbar_warp(&empty[s], phase, abort)) {
                    gave_up(abort, a.status);
                    break;
                }
                if (lane == 0) mbar_arrive(&full[s]);
                ++issued;
                if (++s == C::kStages) {
                    s = 0;
                    phase ^= 1;
                }
            }
        }
        // With many items only now: the merge's CTAs beside this one's start took it 2,000 cycles and more (23 ragged
        // rows of head_dim 64: 20.8 us against 19.8).  With few it is better early (four rows of 256 tokens: 7.3 us
        // against 8.4).
        if (!direct) pdl_launch_dependents();
        if (*abort && lane == 0) {  // leave no copy in flight behind
            for (int i = max(0, issued - C::kStages); i < issued; ++i) {
                const long long t0 = clock64();
                while (!mbar_try_wait(&full[i % C::kStages], (i / C::kStages) & 1) && clock64() - t0 < kWaitTimeoutCycles) {
                }
            }
        }
        return;
    }

    if (warp == kQuery) {
        // ---- items and their queries.  Neighbours of one row group and KV head share them; the first item's are the
        // consumers' work
        uint32_t phase = 1;
        bool fresh = false;
        if (more) named_bar_sync(2, 32 * (kConsumers + 1));
        for (; more; more = w.next<kCols>(a, lane)) {
            if (w.bad && w.part == 0 && lane == 0) report(a.status, DSA_ERR_BOUNDS);
            // the first 16 columns are loaded while the consumers still have the item before
            constexpr int kTurns = 16 / Turn::kTurnCols;
            Turn turns[kTurns];
            auto load = [&](int c0) {
#pragma unroll
                for (int i = 0; i < kTurns; ++i) turns[i].load(a, w, c0 + i * Turn::kTurnCols, cols, hpg, lane);
            };
            if (fresh) load(0);
            if (!wait_mbar_warp(q_empty, phase, abort)) return gave_up(abort, a.status);
            phase ^= 1;
#pragma unroll 1
            for (int c = 0; c < kCols && fresh; c += 16) {
#pragma unroll
                for (int i = 0; i < kTurns; ++i)
                    turns[i].template put<kFp8>(smem + C::OFF_Q, cols_s, a, w, c + i * Turn::kTurnCols, cols, hpg, lane);
                if (c + 16 < kCols) load(c + 16);
            }
            // the item after this one: a part more of the same row group and KV head?
            fresh = !(w.part + 1 < w.parts && w.start + kItemCost + ((w.t_end - w.t_begin + 127) >> 7) < w.end);
            if (lane < 8) item_s->ctx[lane] = w.my_ctx;
            if (lane == 0) {
                item_s->live = 1;
                item_s->t_begin = w.t_begin;
                item_s->t_end = w.t_end;
                item_s->ctx_min = w.ctx_min;
                item_s->row0 = w.row0;
                item_s->g = w.g | (w.col0 << 16);
                item_s->part = w.part;
                item_s->parts = w.parts;
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(q_full);
        }
        if (!wait_mbar_warp(q_empty, phase, abort)) return gave_up(abort, a.status);
        if (lane == 0) {
            item_s->live = 0;
            mbar_arrive(q_full);
        }
        return;
    }

    // ---- consumers
    if (more) {
#pragma unroll 1
        for (int n = warp * Turn::kTurnCols; n < kCols; n += kConsumers * Turn::kTurnCols) {
            Turn t;
            t.load(a, w, n, cols, hpg, lane);
            t.template put<kFp8>(smem + C::OFF_Q, cols_s, a, w, n, cols, hpg, lane);
        }
        asm volatile("bar.arrive 2, %0;" ::"n"(32 * (kConsumers + 1)) : "memory");
    }
    const int cw = warp % kColWarps, tw = warp / kColWarps;
    int s = 0;
    uint32_t phase = 0, q_phase = 0;
    for (;; q_phase ^= 1) {
        if (!wait_mbar_warp(q_full, q_phase, abort)) return gave_up(abort, a.status);
        if (item_s->live == 0) return;
        const int t_begin = item_s->t_begin, t_end = item_s->t_end, ctx_min = item_s->ctx_min;
        const int row0 = item_s->row0, g = item_s->g & 0xffff, col0 = (item_s->g >> 16) + 16 * cw;
        const int part = item_s->part, parts = item_s->parts;
        uint4 q[KS];
        {
            // matrices: columns 0-7, 8-15 of unit 2 k, then of unit 2 k + 1
            const uint32_t qs = smem_u32(smem + C::OFF_Q + cw * C::kQBytes);
#pragma unroll
            for (int k = 0; k < KS; ++k) {
                uint32_t r[4];
                ldsm4(r, qs + q_unit_at<D>(lane & 15, 2 * k + (lane >> 4)));
                q[k] = make_uint4(r[0], r[1], r[2], r[3]);
            }
        }
        float scale[2];
        int cx[2];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            const float2 v = cols_s[16 * cw + gi + 8 * x];
            scale[x] = v.x;
            cx[x] = __float_as_int(v.y);
        }
        // the rows of the group among this warp's columns, and lane i's the context of row i
        const int row_lo = row_of(a, col0), row_hi = row_of(a, min(col0 + 15, cols - 1));
        const int row_ctx = item_s->ctx[lane & 7];
        const bool idle = col0 >= cols;
        __syncwarp();
        if (lane == 0) mbar_arrive(q_empty);

        float o[KS][NT][4] = {};
        float base[2] = {-INFINITY, -INFINITY}, sum[2] = {0.f, 0.f};
        for (int tile0 = t_begin; tile0 < t_end; tile0 += C::kTile) {
            if (!wait_mbar_warp(&full[s], phase, abort)) return gave_up(abort, a.status);
            const uint32_t ks = smem_u32(smem + s * C::kStageBytes), vs = ks + C::kSide;
#pragma unroll 1
            for (int ts = tw * C::kWarpTokens; ts < (tw + 1) * C::kWarpTokens && !idle; ts += C::kStepTokens) {
                const int t0 = tile0 + ts;  // the step's first token
                if (t0 >= t_end) break;
                // S: columns gi, gi + 8; tokens t0 + 8 n + 2 ji + {0, 1}.  ldmatrix brings tokens 0-7
                // (units u, u + 1), then tokens 8-15 of each 16
                float c[2 * SUB][4] = {};
                {
                    const int t = ts + (lane & 7) + ((lane >> 4) << 3), u = (lane >> 3) & 1;
#pragma unroll
                    for (int k = 0; k < KS; k += kFp8 ? 2 : 1) {
#pragma unroll
                        for (int y = 0; y < SUB; ++y) {
                            uint32_t b[4];
                            ldsm4(b, ks + unit_at<C>(t + 16 * y, (kFp8 ? k : 2 * k) + u));
                            if constexpr (!kFp8) {
                                mma16<false>(c[2 * y], q[k], b[0], b[1]);
                                mma16<false>(c[2 * y + 1], q[k], b[2], b[3]);
                            } else {
#pragma unroll
                                for (int n = 0; n < 2; ++n) {
                                    uint32_t b0, b1;
                                    e4m3x4_to_f16(b[2 * n], b0, b1);
                                    mma16<true>(c[2 * y + n], q[k], b0, b1);
                                    e4m3x4_to_f16(b[2 * n + 1], b0, b1);
                                    mma16<true>(c[2 * y + n], q[k + 1], b0, b1);
                                }
                            }
                        }
                    }
                }
                const bool edge = t0 + C::kStepTokens > ctx_min;  // some column does not see all of the step
                if (edge) {
#pragma unroll
                    for (int n = 0; n < 2 * SUB; ++n)
#pragma unroll
                        for (int x = 0; x < 4; ++x)
                            if (t0 + 8 * n + 2 * ji + (x & 1) >= cx[x >> 1]) c[n][x] = -INFINITY;
                }
                float top[2];
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    top[x] = fmaxf(c[0][2 * x], c[0][2 * x + 1]);
#pragma unroll
                    for (int n = 1; n < 2 * SUB; ++n) top[x] = fmaxf(top[x], fmaxf(c[n][2 * x], c[n][2 * x + 1]));
                    top[x] *= scale[x];  // (a positive factor)
                }
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
                    const float b = base[x] == -INFINITY ? 0.f : -base[x];
#pragma unroll
                    for (int n = 0; n < 2 * SUB; ++n)
#pragma unroll
                        for (int y = 0; y < 2; ++y) {
                            c[n][2 * x + y] = ex2(fmaf(c[n][2 * x + y], scale[x], b));
                            sum[x] += c[n][2 * x + y];
                        }
                }
                // P^T as the second product's B operand: n-tile x holds columns 8 x + gi
                uint32_t hi[2 * SUB][NT], lo[2 * SUB][NT];
#pragma unroll
                for (int n = 0; n < 2 * SUB; ++n)
#pragma unroll
                    for (int x = 0; x < NT; ++x) {
                        const float p0 = c[n][2 * x], p1 = c[n][2 * x + 1];
                        if constexpr (kFp8) {
                            hi[n][x] = pack_f16(p0, p1);
                        } else {
                            split_weights(p0, p1, hi[n][x], lo[n][x]);
                        }
                    }
                // O^T += V^T P^T.  In an edge step the rows of the group take turns, with V's tokens at and past
                // the row's context zeroed and the other rows' columns put back: what a row does not see
                // may be NaN, and 0 x NaN must not reach its sums.
                auto product = [&](auto edge_step, int row) {
                    constexpr bool kEdge = decltype(edge_step)::value;
                    uint32_t keep[2 * SUB];  // tokens 8 n + 2 ji + {0, 1}
                    bool mine[NT][2];        // columns 8 x + 2 ji + {0, 1} are this row's
                    if constexpr (kEdge) {
                        const int n_ctx = __shfl_sync(0xffffffffu, row_ctx, row);
#pragma unroll
                        for (int n = 0; n < 2 * SUB; ++n) {
                            const int t = t0 + 8 * n + 2 * ji;
                            keep[n] = (t < n_ctx ? 0xffffu : 0u) | (t + 1 < n_ctx ? 0xffff0000u : 0u);
                        }
#pragma unroll
                        for (int x = 0; x < NT; ++x)
#pragma unroll
                            for (int y = 0; y < 2; ++y)
                                mine[x][y] = static_cast<uint32_t>(col0 + 8 * x + 2 * ji + y - row * hpg) <
                                             static_cast<uint32_t>(hpg);
                    }
                    auto accumulate = [&](float(&acc)[NT][4], uint4 v, int y) {  // 16 tokens y of the step
                        if constexpr (kEdge) {
                            v.x &= keep[2 * y];
                            v.y &= keep[2 * y];
                            v.z &= keep[2 * y + 1];
                            v.w &= keep[2 * y + 1];
                        }
#pragma unroll
                        for (int x = 0; x < NT; ++x) {
                            float old[4];
#pragma unroll
                            for (int z = 0; z < 4; ++z) old[z] = acc[x][z];
                            mma16<kFp8>(acc[x], v, hi[2 * y][x], hi[2 * y + 1][x]);
                            if constexpr (!kFp8) mma16<false>(acc[x], v, lo[2 * y][x], lo[2 * y + 1][x]);
                            if constexpr (kEdge) {
#pragma unroll
                                for (int z = 0; z < 4; ++z) acc[x][z] = mine[x][z & 1] ? acc[x][z] : old[z];
                            }
                        }
                    };
#pragma unroll
                    for (int y = 0; y < SUB; ++y) {
                        if constexpr (!kFp8) {
                            // matrices: tokens 0-7 (d 0-7, 8-15), tokens 8-15 (d 0-7, 8-15)
                            const int t = ts + 16 * y + (lane & 7) + ((lane >> 4) << 3), u = (lane >> 3) & 1;
#pragma unroll
                            for (int m = 0; m < KS; ++m) {
                                uint32_t v[4];
                                ldsm4_t(v, vs + unit_at<C>(t, 2 * m + u));
                                accumulate(o[m], make_uint4(v[0], v[1], v[2], v[3]), y);
                            }
                        } else {
                            // matrices: unit m tokens 0-7, 8-15, unit m + 1 likewise; a lane gets codes
                            // [t d][t d+1][t+1 d][t+1 d+1], d = 2 gi: M row gi is dim 2 gi, row gi + 8 dim 2 gi + 1
                            const int t = ts + 16 * y + (lane & 15), u = lane >> 4;
#pragma unroll
                            for (int m = 0; m < KS; m += 2) {
                                uint32_t w[4];
                                ldsm4_t(w, vs + unit_at<C>(t, m + u));
#pragma unroll
                                for (int z = 0; z < 2; ++z) {
                                    uint4 v;
                                    e4m3x4_to_f16(__byte_perm(w[2 * z], 0, 0x3120), v.x, v.y);
                                    e4m3x4_to_f16(__byte_perm(w[2 * z + 1], 0, 0x3120), v.z, v.w);
                                    accumulate(o[m + z], v, y);
                                }
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
            if (++s == C::kStages) {
                s = 0;
                phase ^= 1;
            }
        }
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            sum[x] += __shfl_xor_sync(0xffffffffu, sum[x], 1);
            sum[x] += __shfl_xor_sync(0xffffffffu, sum[x], 2);
        }

        // ---- output
        auto place_of = [&](int col) {  // row * num_heads + head
            const int row = row_of(a, col);
            return static_cast<int64_t>(row0 + row) * a.num_heads + g * hpg + col - row * hpg;
        };
        auto finish = [&](int64_t at, int d, const float4 &x, float b, float total) {  // dims d .. d + 3 of head `at`
            if (parts > 1) {
                *reinterpret_cast<float4 *>(a.part_o + (at * a.parts_bound + part) * D + d) = x;
                if (d == 0) a.part_ml[at * a.parts_bound + part] = make_float2(part_base(b, total), total);
            } else {
                const bool none = total == 0.f;
                const float inv = none ? 0.f : a.v_scale / total;
                *reinterpret_cast<uint2 *>(a.out + at * D + d) =
                    none ? make_uint2(0u, 0u) : make_uint2(pack_bf16(x.x * inv, x.y * inv), pack_bf16(x.z * inv, x.w * inv));
                if (d == 0 && a.lse != nullptr) a.lse[at] = none ? -INFINITY : (b + log2f(total)) * 0.6931471805599453f;
            }
        };
        if constexpr (kTokWarps > 1) {
            // the token warps' outputs meet in the next stage of the ring, each in its own base; every consumer
            // then adds up its share of the columns, token warps in order
            if (!wait_mbar_warp(&full[s], phase, abort)) return gave_up(abort, a.status);
            float *mo = reinterpret_cast<float *>(smem + s * C::kStageBytes);
            float *mine = mo + warp * C::kMergeFloats;
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int y = 0; y < 2; ++y)
#pragma unroll
                    for (int m = 0; m < KS; ++m) {
                        const int c = 8 * n + 2 * ji + y;
                        if constexpr (kFp8) {  // dims 16 m + 2 gi, 2 gi + 1
                            *reinterpret_cast<float2 *>(mine + merge_at<D>(c, 16 * m + 2 * gi)) =
                                make_float2(o[m][n][y], o[m][n][2 + y]);
                        } else {               // dims 16 m + gi, gi + 8
                            mine[merge_at<D>(c, 16 * m + gi)] = o[m][n][y];
                            mine[merge_at<D>(c, 16 * m + gi + 8)] = o[m][n][2 + y];
                        }
                    }
            // (two sets: a warp may be an item ahead of one that still reads)
            float2 *ml = ml_s + q_phase * (kConsumers * 16);
            if (ji == 0) {
                ml[warp * 16 + gi] = make_float2(base[0], sum[0]);
                ml[warp * 16 + gi + 8] = make_float2(base[1], sum[1]);
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(merge);
            if (!wait_mbar_warp(merge, q_phase, abort)) return gave_up(abort, a.status);
            constexpr int kLanes = D / 4;  // lanes of a column
            const int first = warp * (32 / kLanes) + lane / kLanes, d = lane % kLanes * 4;
            const int here = min(kCols, cols - (col0 - 16 * cw));
#pragma unroll 2
            for (int n = first; n < here; n += kConsumers * (32 / kLanes)) {
                float b = -INFINITY;
#pragma unroll
                for (int w = 0; w < kTokWarps; ++w) b = fmaxf(b, ml[(w * kColWarps + n / 16) * 16 + n % 16].x);
                const float b0 = b == -INFINITY ? 0.f : b;
                float total = 0.f;
                float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int w = 0; w < kTokWarps; ++w) {
                    const int from = w * kColWarps + n / 16;
                    const float2 l = ml[from * 16 + n % 16];
                    const float4 y = *reinterpret_cast<const float4 *>(mo + from * C::kMergeFloats + merge_at<D>(n % 16, d));
                    const float f = ex2(l.x - b0);
                    total += l.y * f;
                    x.x += y.x * f;
                    x.y += y.y * f;
                    x.z += y.z * f;
                    x.w += y.w * f;
                }
                const int col = col0 - 16 * cw + n;
                finish(place_of(col), d, x, b0, total);
            }
            fence_async_smem();  // the stage goes back to TMA writes
            __syncwarp();
            if (lane == 0) mbar_arrive(&empty[s]);
            if (++s == C::kStages) {
                s = 0;
                phase ^= 1;
            }
        } else {
            // one warp has all of a column: lanes swap dims so that each writes four in a row
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    const float b = __shfl_sync(0xffffffffu, base[n], 8 * ji + 4 * y);
                    const float total = __shfl_sync(0xffffffffu, sum[n], 8 * ji + 4 * y);
                    const int col = col0 + 8 * n + 2 * ji + y;
                    const int64_t at = place_of(col);
#pragma unroll
                    for (int m = 0; m < KS; ++m) {
                        // own: dims {p, q}; FP8: 2 gi, 2 gi + 1 of 16 m; else gi, gi + 8
                        float p = o[m][n][y], q2 = o[m][n][2 + y];
                        if constexpr (kFp8) {
                            const float r0 = __shfl_xor_sync(0xffffffffu, p, 4), r1 = __shfl_xor_sync(0xffffffffu, q2, 4);
                            if ((gi & 1) == 0 && col < cols)
                                finish(at, 16 * m + 2 * gi, make_float4(p, q2, r0, r1), b == -INFINITY ? 0.f : b, total);
                        } else {
                            // even gi collects dims gi, gi + 1 (and, two lanes on, gi + 2, gi + 3), odd gi the upper eight
                            const float give = gi & 1 ? p : q2;
                            const float got = __shfl_xor_sync(0xffffffffu, give, 4);
                            const float e0 = gi & 1 ? got : p, e1 = gi & 1 ? q2 : got;  // dims 2 (gi / 2), + 1 of its eight
                            const float f0 = __shfl_xor_sync(0xffffffffu, e0, 8), f1 = __shfl_xor_sync(0xffffffffu, e1, 8);
                            if ((gi & 2) == 0 && col < cols)
                                finish(at, 16 * m + (gi & 1) * 8 + (gi & 4), make_float4(e0, e1, f0, f1),
                                       b == -INFINITY ? 0.f : b, total);
                        }
                    }
                }
        }
    }
}

// Merge of a row's parts: one CTA per (row, head).  128 / (D / 4) groups of lanes take every so manyth part,
// four dims to a lane; the groups' sums are added in order.
constexpr int kCombineThreads = 128, kCombineParts = 128;

template <int D>
__global__ void __launch_bounds__(kCombineThreads) kv_combine_kernel(const __grid_constant__ KvAttnArgs a) {
    constexpr int kLanes = D / 4, kGroups = kCombineThreads / kLanes;
    __shared__ float2 ml_s[kCombineParts];
    __shared__ float4 x_s[kGroups][kLanes];
    __shared__ float t_s[kGroups];
    // The attention kernel lets this one start after its own wait, so what ran before it is complete: the
    // contexts can be read before this kernel's wait, which is for the parts.  (A refused group is one part.)
    const int64_t at = blockIdx.x;
    int req;
    bool bad;
    const int my_ctx = kv_load_group(a, static_cast<int>(at / a.num_heads) / a.group * a.group, threadIdx.x & 31, req, bad);
    const int ctx = __reduce_max_sync(0xffffffffu, my_ctx);
    const int parts = kv_parts(ctx, kv_part_shift(ctx, a.parts_shift));
    pdl_wait();
    pdl_launch_dependents();
    if (parts == 1) return;  // written by the attention kernel
    const int grp = threadIdx.x / kLanes, d = threadIdx.x % kLanes;
    const float4 *po = reinterpret_cast<const float4 *>(a.part_o + at * a.parts_bound * D) + d;
    // the first parts' outputs are on their way while the bases are compared
    constexpr int kAhead = 8;
    float4 y[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
        const int p = grp + i * kGroups;
        if (p < parts) y[i] = po[static_cast<int64_t>(p) * kLanes];
    }
    for (int p = threadIdx.x; p < parts; p += kCombineThreads) ml_s[p] = a.part_ml[at * a.parts_bound + p];
    __syncthreads();
    float b = -INFINITY;
    for (int p = threadIdx.x & 31; p < parts; p += 32) b = fmaxf(b, ml_s[p].x);
#pragma unroll
    for (int i = 16; i > 0; i >>= 1) b = fmaxf(b, __shfl_xor_sync(0xffffffffu, b, i));
    const float b0 = b == -INFINITY ? 0.f : b;
    float total = 0.f;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    auto add = [&](int p, const float4 &v) {
        const float2 l = ml_s[p];
        const float f = ex2(l.x - b0);
        total += l.y * f;
        x.x += v.x * f;
        x.y += v.y * f;
        x.z += v.z * f;
        x.w += v.w * f;
    };
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
        if (grp + i * kGroups < parts) add(grp + i * kGroups, y[i]);
#pragma unroll 4
    for (int p = grp + kAhead * kGroups; p < parts; p += kGroups) add(p, po[static_cast<int64_t>(p) * kLanes]);
    x_s[grp][d] = x;
    if (d == 0) t_s[grp] = total;
    __syncthreads();
    if (grp > 0) return;
#pragma unroll
    for (int i = 1; i < kGroups; ++i) {
        const float4 v = x_s[i][d];
        x.x += v.x;
        x.y += v.y;
        x.z += v.z;
        x.w += v.w;
        total += t_s[i];
    }
    const bool none = total == 0.f;
    const float inv = none ? 0.f : a.v_scale / total;
    *reinterpret_cast<uint2 *>(a.out + at * D + 4 * d) =
        none ? make_uint2(0u, 0u) : make_uint2(pack_bf16(x.x * inv, x.y * inv), pack_bf16(x.z * inv, x.w * inv));
    if (d == 0 && a.lse != nullptr) a.lse[at] = none ? -INFINITY : (b0 + log2f(total)) * 0.6931471805599453f;
}

template <bool kFp8, int D, bool kWide, int kColWarps>
cudaError_t launch_variant(KvAttnArgs &a, cudaStream_t s) {
    using C = KvCfg<kFp8, D, kColWarps>;
    auto kern = kv_attention_kernel<kFp8, D, kWide, kColWarps>;
    static std::atomic<uint64_t> configured{0};
    cudaError_t e = raise_smem_limit(kern, C::kSmemBytes, configured);
    if (e != cudaSuccess) return e;
    CUtensorMap map;
    if (!encode_kv_rows_map(&map, a.pool, a.pool_rows, C::kRowBytes, a.page_size < C::kTile ? a.page_size : C::kTile))
        return cudaErrorInvalidValue;
    const uint32_t ctas = persistent_ctas(a);
    if (ctas == 0) return cudaErrorInvalidDevice;
    return launch_pdl(kern, dim3(ctas), dim3(kThreads), C::kSmemBytes, s, map, a);
}

template <bool kFp8, int D>
cudaError_t launch_format(KvAttnArgs &a, cudaStream_t s) {
    const int cols = a.group * (a.num_heads / a.kv_heads);
    const int col_warps = cols <= 16 ? 1 : cols <= 32 ? 2 : 4;
    a.col_blocks = (cols + 16 * col_warps - 1) / (16 * col_warps);
    const int64_t items = static_cast<int64_t>(a.num_rows / a.group) * a.kv_heads * a.col_blocks * a.parts_bound;
    if (items > 0x7fffffff) return cudaErrorInvalidConfiguration;
    a.items = static_cast<uint32_t>(items);
    if (cols <= 8) return launch_variant<kFp8, D, false, 1>(a, s);
    if (col_warps == 1) return launch_variant<kFp8, D, true, 1>(a, s);
    if (col_warps == 2) return launch_variant<kFp8, D, true, 2>(a, s);
    return launch_variant<kFp8, D, true, 4>(a, s);
}

}  // namespace

size_t kv_attention_workspace_bytes(int64_t num_rows, int32_t num_heads, int32_t kv_heads, int32_t head_dim,
                                    int32_t max_ctx) {
    const size_t parts = static_cast<size_t>(kv_parts_bound(max_ctx, kv_parts_shift(kv_heads)));
    if (parts <= 1) return 0;
    const size_t n = static_cast<size_t>(num_rows) * static_cast<size_t>(num_heads) * parts;
    return align256(n * static_cast<size_t>(head_dim) * 4) + align256(n * 8);
}

cudaError_t launch_kv_attention(KvAttnArgs &a, void *workspace, cudaStream_t s) {
    if (a.num_rows == 0) return cudaSuccess;
    for (a.page_shift = 4; 1 << a.page_shift < a.page_size;) ++a.page_shift;
    const uint32_t hpg = static_cast<uint32_t>(a.num_heads / a.kv_heads);
    a.hpg = static_cast<int32_t>(hpg);
    a.hpg_mul = ((1u << 20) + hpg - 1) / hpg;
    a.parts_shift = kv_parts_shift(a.kv_heads);
    a.parts_bound = kv_parts_bound(a.max_ctx, a.parts_shift);
    const size_t n = static_cast<size_t>(a.num_rows) * static_cast<size_t>(a.num_heads) * a.parts_bound;
    a.part_o = static_cast<float *>(workspace);
    a.part_ml = reinterpret_cast<float2 *>(static_cast<uint8_t *>(workspace) +
                                           align256(n * static_cast<size_t>(a.head_dim) * 4));
    cudaError_t e;
    if (a.fp8) e = a.head_dim == 64 ? launch_format<true, 64>(a, s) : launch_kv_attention_fp8(a, s);
    else e = a.head_dim == 64 ? launch_format<false, 64>(a, s) : launch_format<false, 128>(a, s);
    if (e != cudaSuccess || a.parts_bound == 1) return e;
    const int64_t grid = static_cast<int64_t>(a.num_rows) * a.num_heads;
    if (grid > 0x7fffffff) return cudaErrorInvalidConfiguration;
    const dim3 gr(static_cast<unsigned>(grid)), b(kCombineThreads);
    return a.head_dim == 64 ? launch_pdl(kv_combine_kernel<64>, gr, b, 0, s, a)
                            : launch_pdl(kv_combine_kernel<128>, gr, b, 0, s, a);
}

}  // namespace dsa
