// kv_attention_fp8.cu -- dense attention over a paged FP8 K/V pool of head_dim 128 (dsa_kv_attention).
//
//   out[r, h, :] = sum_t softmax_t(sm_scale <q[r,h,:], K_g,t>) V_g,t   over t < row_ctx[r]
//
// An FP8 token of a KV head is 256 bytes, so the bytes leave half the time of a bf16 one per column, and
// warp-level MMAs, which need the codes as fp16 fragments, do not keep up (kv_attention.cu: 32 x 16K-64K
// tokens in 327 us against 203 us at the copy bandwidth, nothing but conversions and issue slots in the
// way; here 222 us).  The fifth-generation tensor cores take the codes as they lie in shared memory:
//
//     S^T[128 tokens x NC]  = K Q^T      A: the K tile (K-major), B: q as hi, then lo e4m3 terms
//     O^T[128 dims x NC]   += V^T P^T    A: the V tile read MN-major, B: P as three e5m2 terms (MN-major)
//
// with NC (16, 32 or 64) columns, (row of the group, query head of the KV head) pairs, in N.  An MMA with so
// small an N costs its A operand's passage: 40 cycles an SM for N <= 32, 48 for 64, 64 for 128 measured, so a tile's
// 8, 12 or 16 take some 340 to 830 of the 1,490 cycles that its 32 KB take at the copy bandwidth.  A token is a TMEM
// lane: a softmax thread reads its token's scores of its columns, P = 2^(S - b) with a lazy base b per column, splits
// each weight into three terms and writes its row of P.  The base moves, and O^T is rescaled in TMEM, only when a
// score exceeds it by 2^15.7.
//
// Roles: softmax warps (TMEM lane quadrants; one warpgroup, or two that share out 64 columns), a TMA producer
// (K and V tiles of 16 KB through a ring each), an issuer of the scores' MMAs, one of the values' (an MMA's
// issue lasts as long as its passage, so one thread for both would set the pace), a query warp (items and
// their query images).  Two persistent CTAs per SM take equal shares of the items (row group, KV head, column
// block, part of the context; kv_attention_common.cuh); parts are merged by kv_combine_kernel
// (kv_attention.cu).
//
// What bounds it: for 16 columns the bytes once contexts are long (32 x 16K-64K: 222 us, 91% of the copy
// bandwidth; tiles of one CTA follow each other in 1,200 cycles when the memory lets them, an item costs about 4,000
// cycles more: its first base, the last product's passage, its output).  Short parts show that, and the 5,000
// cycles from the launch to the first tile (24 x 8K: 50 us against 30 us of bytes).  Writing an item's output behind
// the next one's first weights, into a second buffer of outputs, was slower (51 us): the other CTA of the SM fills the
// wait already.  For 64 columns a tile takes some 4,000 cycles, most of them the softmax warps' latencies (fewer than
// half of the issue slots are used), and a verify step of 4 x 64K tokens and 4 x 16 columns 92 us against 38 us of
// bytes.  (When it took 99: two blocks of 32 columns, which read the cache twice, 126 us, one warpgroup for all 64
// columns 172 us, sums of weights in registers, which then spill, 106 us.)  P's third term costs 3 to 4 us of the 92;
// all three one after the other into one accumulator, with a second score buffer in the place of the other, 102 us.
//
// Precision: products of two 8-bit numbers are exact and accumulate in fp32.  q is scaled by a power of two per
// column and written as hi + lo (exact but for elements 2^-9 below the column's largest, which are within 2^-17 of
// it).  A weight is rounded to fp16 (2^-11 of itself at worst, against the output's own 2^-8), whose 11 bits three
// e5m2 terms of 3 hold exactly; e5m2's smallest step is 2^-16 and the largest weight at least 2^13, so weights keep
// 2^-29 of their part's largest: the background behind an attention sink counts, however many tokens make it up.
// (Two e4m3 terms over a largest of 2^6 lost what lay 2^16 below it: with a first token 11 nats ahead of 131,072
// others, whose values it opposes, an output of +0.26 for +0.30.)
#include "kv_attention_common.cuh"
#include "mla_fp8_common.cuh"

namespace dsa {

namespace {

using namespace kv;
using fp8mla::split_pair;
using fp8mla::sw128;

constexpr int kTile = 128;                                 // tokens of a tile
constexpr int kDim = 128;
constexpr int kUnitBytes = kTile * kDim;                   // K or V of a tile
constexpr float kTop = 15.7f;                              // weights reach 2^15.7 = 53,232 (e5m2 holds 57,344) ...
constexpr float kBias = 13.0f;                             // ... and a moved base leaves the largest at 2^13

// What the query warp tells the others about an item.
struct Item {
    int32_t live;              // 0: no more items
    int32_t t_begin, t_end;
    int32_t ctx_min, ctx_max;  // over the rows of the group
    int32_t cols;              // real columns
    int32_t part, to_parts;    // (whether its output goes to the workspace)
    int32_t ctx[8];            // the group's contexts
    int32_t image_last;        // the next item has another query image
    int32_t pad[15];
};
static_assert(sizeof(Item) == 128, "item layout");

// An item's columns: log2 units per unit of score, tokens seen, row * num_heads + head.
template <int NC>
struct Columns {
    float scale[NC];
    int32_t ctx[NC], at[NC];
};

template <int NC>
struct Cfg {
    // K and V tiles go through rings of their own, so that whoever waits for a tile has waited for every one before
    // it in its slot (a barrier's parity alone cannot tell a phase from the one two before it)
    static constexpr int kK = 2, kV = NC == 16 ? 3 : 2, kUnits = kK + kV;
    static constexpr int kQBytes = 2 * NC * kDim, kQBufs = NC == 64 ? 1 : 2;
    // Softmax warpgroups, each with its share of the columns, and the four other warps behind them.
    static constexpr int kGroups = NC == 64 ? 2 : 1, kMine = NC / kGroups;
    static constexpr int kSoftmax = 4 * kGroups;
    static constexpr int kProducer = kSoftmax, kScores = kSoftmax + 1, kQuery = kSoftmax + 2, kValues = kSoftmax + 3;
    static constexpr int kThreads = 32 * (kSoftmax + 4);
    // Registers a thread: at launch (two CTAs fill the SM), then the softmax warpgroups take some of the others'.
    static constexpr int kLaunchRegs = kGroups == 1 ? 128 : 80;
    static constexpr int kSoftmaxRegs = kGroups == 1 ? 168 : 88, kOtherRegs = kGroups == 1 ? 88 : 64;
    static_assert(kGroups * kSoftmaxRegs + kOtherRegs == (kGroups + 1) * kLaunchRegs,
                  "the warpgroups share what the CTA was launched with");
    // A product's terms lie side by side in an MMA's N, each with its accumulator, or follow one another into one: q's
    // hi and lo for 16 columns, else one after the other; P's three, but for 64 columns the third after the first
    static constexpr int kSN = NC == 16 ? 2 * NC : NC, kON = NC == 64 ? 2 * NC : 3 * NC;
    static constexpr int kSTurns = NC == 16 ? 1 : 2, kOTurns = NC == 64 ? 2 : 1;
    static constexpr int kSBufs = NC == 64 ? 1 : 2, kPBufs = NC == 16 ? 2 : 1;
    // P: a token's 128-byte row holds its three terms (64 columns: the first two) of each buffer; the third terms of
    // 64 columns have rows of 64 bytes, tokens 64 and up beside the first 64 in 128
    static constexpr int kPRow = (NC == 64 ? 2 : 3) * NC / 16;  // 16-byte units of a buffer in a token's row
    static constexpr int kP3Bytes = NC == 64 ? kTile * 64 : 0;
    static constexpr uint32_t kP3Offset = kTile * 128 / 16;     // units from P's rows to the third terms'
    // (a softmax warp that waits for a V tile alone, on an edge, has seen the product of the tile kPBufs before: the
    // barrier's phase before the awaited one is over)
    static_assert(kPBufs <= kV, "a V tile's phases are told apart");
    static constexpr bool kSumsInTmem = NC == 64;          // a thread's sums of weights, if not in registers
    static constexpr uint32_t kTmemO = kSBufs * kSN;       // score buffers, then the output, then the sums
    static constexpr uint32_t kTmemL = kTmemO + kON;
    static constexpr uint32_t kTmemCols = 256;             // two CTAs share the SM's 512
    // where a product for the columns of one context of a group goes: of 64 columns into the scores' buffer, one of
    // O^T's two accumulators at a time
    static constexpr bool kApartInScores = NC == 64;
    static constexpr int kApartTurns = kApartInScores ? 2 : 1, kXN = kON / kApartTurns;
    static constexpr uint32_t kTmemX = kApartInScores ? 0 : kTmemL;
    static constexpr int OFF_Q = kUnits * kUnitBytes;      // [kQBufs]: rows hi 0 .. NC - 1, lo NC .. 2 NC - 1
    static constexpr int OFF_P = OFF_Q + kQBufs * kQBytes;
    static constexpr int OFF_P3 = OFF_P + kTile * 128;
    static constexpr int OFF_SCHED = OFF_P;                // of use before the first weights alone
    static constexpr int OFF_COLS = OFF_P3 + kP3Bytes;     // [2] by image parity
    static constexpr int OFF_ITEM = OFF_COLS + 2 * static_cast<int>(sizeof(Columns<NC>));
    static constexpr int OFF_MAX = OFF_ITEM + 2 * static_cast<int>(sizeof(Item));      // [kSoftmax][kMine] a warp's largest scores
    static constexpr int OFF_BASE = OFF_MAX + 4 * NC * 4;  // [kSoftmax][kMine] minus the bases, a copy per warp
    static constexpr int OFF_FAC = OFF_BASE + 4 * NC * 4;  // [kSoftmax][kMine] rescale factors
    static constexpr int OFF_MOVE = OFF_FAC + 4 * NC * 4;  // [kSoftmax][kMine] and their logarithms
    static constexpr int OFF_SUM = OFF_MOVE + 4 * NC * 4;   // [2][kSoftmax][kMine] sums of weights, by item parity
    static constexpr int OFF_BARS = OFF_SUM + 2 * 4 * NC * 4;
    static constexpr int kNumBars = 2 * kUnits + 2 * 2 + 2 * 2 + kQBufs + 2 * kPBufs + 2;
    static constexpr int OFF_MISC = OFF_BARS + kNumBars * 8;
    static constexpr int kSmemBytes = OFF_MISC + 16 + 1024;
    static_assert(sizeof(KvSchedule) <= kTile * 128, "the schedule fits P");
    static_assert(kTmemL + (kSumsInTmem ? NC : 0) + (kApartInScores ? 0 : kXN) <= kTmemCols, "TMEM plan");
    static_assert(kApartInScores ? kXN <= kSN : !kSumsInTmem, "TMEM plan");
    static_assert(kSmemBytes <= 115712, "two CTAs per SM");
};

// Sums over the warp's lanes of v[0..N): afterwards v[0] of lane l belongs to column
// lane_column<N>(l).  Halves of the columns change hands, so N columns take N shuffles (N = 16: 16, 32: 31).
template <int N>
__device__ __forceinline__ void reduce_lanes(float (&v)[N], int lane) {
    int n = N;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
        if (n > 1) {
            n >>= 1;
            const bool up = (lane & off) != 0;
#pragma unroll
            for (int i = 0; i < N / 2; ++i) {
                if (i >= n) break;
                v[i] = (up ? v[i + n] : v[i]) + __shfl_xor_sync(0xffffffffu, up ? v[i] : v[i + n], off);
            }
        } else {
            v[0] += __shfl_xor_sync(0xffffffffu, v[0], off);
        }
    }
}

template <int N>
__device__ __forceinline__ int lane_column(int lane) {
    static_assert(N == 16 || N == 32, "");
    return N == 32 ? lane : lane >> 1;
}

// The columns' sums over the warp's tokens into dst[0..N).
template <int N>
__device__ __forceinline__ void reduce_columns(float (&v)[N], float *dst, int lane) {
    reduce_lanes<N>(v, lane);
    if (N == 32 || (lane & 1) == 0) dst[lane_column<N>(lane)] = v[0];
}

// The columns' maxima over the warp's tokens into dst[0..N); a NaN is passed over.
template <int N>
__device__ __forceinline__ void max_columns(const float (&v)[N], float *dst, int lane) {
#pragma unroll
    for (int j = 0; j < N; j += 4) {
        float m[4];
#pragma unroll
        for (int k = 0; k < 4; ++k)
            asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(m[k]) : "f"(v[j + k]));
        if (lane == 0) *reinterpret_cast<float4 *>(dst + j) = make_float4(m[0], m[1], m[2], m[3]);
    }
}

// (h0, h1) += (g0, g1), fp32.
__device__ __forceinline__ void add_pair(uint32_t &h0, uint32_t &h1, float g0, float g1) {
    const float2 s = __fadd2_rn(make_float2(__uint_as_float(h0), __uint_as_float(h1)), make_float2(g0, g1));
    h0 = __float_as_uint(s.x);
    h1 = __float_as_uint(s.y);
}

// Four weights as fp16 in (a, b): their first, second and third e5m2 terms.  An e5m2 number is the upper byte of an
// fp16 one: each term is what is left, rounded to that byte (half a step up), and the rest is exact.
__device__ __forceinline__ void weight_terms(uint32_t a, uint32_t b, uint32_t &t1, uint32_t &t2, uint32_t &t3) {
    auto rest = [](uint32_t x, uint32_t rounded) {
        const uint32_t byte = rounded & 0xff00ff00u;
        const __half2 d = __hsub2(*reinterpret_cast<const __half2 *>(&x), *reinterpret_cast<const __half2 *>(&byte));
        return *reinterpret_cast<const uint32_t *>(&d);
    };
    uint32_t ra = a + 0x00800080u, rb = b + 0x00800080u;
    t1 = __byte_perm(ra, rb, 0x7531);
    a = rest(a, ra);
    b = rest(b, rb);
    ra = a + 0x00800080u;
    rb = b + 0x00800080u;
    t2 = __byte_perm(ra, rb, 0x7531);
    t3 = __byte_perm(rest(a, ra), rest(b, rb), 0x7531);
}

__device__ __forceinline__ void add16(uint32_t (&h)[16], const uint32_t (&g)[16]) {
#pragma unroll
    for (int j = 0; j < 16; j += 2) add_pair(h[j], h[j + 1], __uint_as_float(g[j]), __uint_as_float(g[j + 1]));
}

// OR of a predicate over the softmax warps (kN threads), who all meet here.
template <int kN>
__device__ __forceinline__ bool meet_any_of(bool p) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
        "barrier.cta.red.or.pred.aligned q, 1, %2, p;\n\tselp.u32 %0, 1, 0, q;\n\t}\n"
        : "=r"(r)
        : "r"(static_cast<uint32_t>(p)), "n"(kN)
        : "memory");
    return r != 0;
}

// Whether any of four e4m3 codes is NaN (0x7f or 0xff).
__device__ __forceinline__ bool any_nan4(uint32_t v) { return __vcmpeq4(v & 0x7f7f7f7fu, 0x7f7f7f7fu) != 0; }

// A column's query as hi and lo terms, and its scale.  The 16 bf16 elements of lane's unit (lane & 7) of column n
// are in v0, v1; the eight lanes of a column work together, so a warp takes four.
template <int NC>
__device__ __forceinline__ void convert_query(uint8_t *img, Columns<NC> *cs, const KvAttnArgs &a, const KvCursor<kEither> &w,
                                              int n, int cols, int hpg, uint4 v0, uint4 v1, int lane) {
    const int unit = lane & 7;
    const uint32_t h[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
    // the column's largest |q| by its bits (an infinity or a NaN is above every number)
    uint32_t top = 0;
#pragma unroll
    for (int y = 0; y < 8; ++y) top = max(top, max(h[y] << 16 & 0x7fff0000u, h[y] & 0x7fff0000u));
#pragma unroll
    for (int y = 1; y < 8; y <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, y));
    const bool finite = top < 0x7f800000u;
    // 2^e brings it to (224, 448]
    int e = 0;
    if (top > 0 && finite) {
        e = 135 - static_cast<int>(top >> 23) - ((top & 0x7fffffu) > 0x600000u ? 1 : 0);
        e = max(-120, min(120, e));
    }
    const float up = __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
    uint32_t hi[4], lo[4];
#pragma unroll
    for (int y = 0; y < 4; ++y) {
        const uint2 p0 = split_pair(bf16_lo(h[2 * y]) * up, bf16_hi(h[2 * y]) * up);
        const uint2 p1 = split_pair(bf16_lo(h[2 * y + 1]) * up, bf16_hi(h[2 * y + 1]) * up);
        hi[y] = p0.x | (p1.x << 16);
        lo[y] = p0.y | (p1.y << 16);
    }
    *reinterpret_cast<uint4 *>(img + sw128(n, unit)) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
    *reinterpret_cast<uint4 *>(img + sw128(NC + n, unit)) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
    const int col = w.col0 + n, row = col < cols ? static_cast<int>(col * a.hpg_mul >> 20) : 0;
    const int ctx = __shfl_sync(0xffffffffu, w.my_ctx, row);
    if (unit == 0) {
        // a masked score is -inf times the scale: neither zero nor infinity.  A NaN or an infinity
        // in q makes its column's scores, and so its output, NaN
        const float scale = a.s_scale * __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
        cs->scale[n] = finite ? fminf(fmaxf(scale, 1.17549435e-38f), 3.40282347e38f) : __uint_as_float(0x7fc00000u);
        cs->ctx[n] = col < cols ? ctx : 0;
        cs->at[n] = (w.row0 + row) * a.num_heads + w.g * hpg + (col < cols ? col - row * hpg : 0);
    }
}

// The 16 elements that convert_query wants of column n; zeros behind the last column.
__device__ __forceinline__ void load_query(const KvAttnArgs &a, const KvCursor<kEither> &w, int n, int cols, int hpg, int lane,
                                           uint4 &v0, uint4 &v1) {
    v0 = v1 = make_uint4(0u, 0u, 0u, 0u);
    const int col = w.col0 + n;
    if (col < cols) {
        const int row = static_cast<int>(col * a.hpg_mul >> 20);
        const uint4 *src = reinterpret_cast<const uint4 *>(a.q + (w.row0 + row) * a.q_stride +
                                                           static_cast<int64_t>(w.g * hpg + col - row * hpg) * kDim +
                                                           (lane & 7) * 16);
        v0 = src[0];
        v1 = src[1];
    }
}

template <int NC>
__global__ void __launch_bounds__(Cfg<NC>::kThreads, 2)
    kv_attention_fp8_kernel(const __grid_constant__ CUtensorMap kv_map, const __grid_constant__ KvAttnArgs a) {
    using C = Cfg<NC>;
    constexpr int kSoftmax = C::kSoftmax, kProducer = C::kProducer, kScores = C::kScores, kQuery = C::kQuery,
                  kValues = C::kValues, kMine = C::kMine;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    Columns<NC> *cols_s = reinterpret_cast<Columns<NC> *>(smem + C::OFF_COLS);
    Item *item_s = reinterpret_cast<Item *>(smem + C::OFF_ITEM);
    float *sum_s = reinterpret_cast<float *>(smem + C::OFF_SUM);
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + C::OFF_BARS);  // [kK + kV] K or V landed
    uint64_t *empty = full + C::kUnits;                                 // [kK + kV] the MMAs that read it are done
    uint64_t *s_full = empty + C::kUnits;                               // [2] scores in TMEM
    uint64_t *s_empty = s_full + 2;                             // [2] softmax has read them
    uint64_t *q_full = s_empty + 2, *q_empty = q_full + 2;      // [2] an item and its columns, by item parity
    uint64_t *img_empty = q_empty + 2;                                  // [kQBufs] the MMAs are done with the queries
    uint64_t *p_full = img_empty + C::kQBufs;                           // [kPBufs] weights written (and O^T rescaled)
    uint64_t *pv_done = p_full + C::kPBufs;                             // [kPBufs] O^T += V^T P^T done
    uint64_t *o_empty = pv_done + C::kPBufs;                            // the item's output is read
    uint64_t *drained = o_empty + 1;                                    // after a wait gave up: no MMA is left
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + C::OFF_MISC);
    volatile int *abort = reinterpret_cast<volatile int *>(smem + C::OFF_MISC + 4);
    volatile int32_t *levels_s = reinterpret_cast<volatile int32_t *>(smem + C::OFF_MISC + 8);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        *abort = 0;
        *levels_s = 0;
        for (int s = 0; s < C::kUnits; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(&s_full[s], 1);
            mbar_init(&s_empty[s], kSoftmax);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(&q_full[s], 1);
            mbar_init(&q_empty[s], kSoftmax + 2);
        }
        for (int s = 0; s < C::kQBufs; ++s) mbar_init(&img_empty[s], 1);
        for (int s = 0; s < C::kPBufs; ++s) {
            mbar_init(&p_full[s], kSoftmax);
            mbar_init(&pv_done[s], 1);
        }
        mbar_init(o_empty, kSoftmax);
        mbar_init(drained, 2);
        fence_mbar_init();
        prefetch_tensormap(&kv_map);
    }
    if (warp == kScores) {
        tmem_alloc(tmem_slot, C::kTmemCols);
        tmem_relinquish();
        tc_fence_before();
    }
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    pdl_wait();
    const bool direct = kv_direct(a);
    if (direct || a.keep_parts) pdl_launch_dependents();
    KvSchedule *sched = reinterpret_cast<KvSchedule *>(smem + C::OFF_SCHED);
    if (!kv_fill_schedule<kEither>(a, sched)) {
        if (warp == kScores) tmem_dealloc(tmem, C::kTmemCols);
        return;
    }
    __syncthreads();

    const int hpg = a.hpg, cols = a.group * hpg;
    KvCursor<kEither> w;
    bool more = w.first<NC>(a, sched, lane);
    if (!direct) __syncthreads();  // the schedule's place is P's

    if (warp >= kSoftmax) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kOtherRegs));
        if (warp == kProducer) {
            // ---- K and V: boxes of at most 128 rows, lane b issues box b of a unit
            const int box_rows = min(a.page_size, kTile);
            const int box_shift = min(a.page_shift, 7), boxes = kTile >> box_shift;
            const uint64_t policy = l2_evict_first_policy();
            uint32_t issued = 0;  // tiles
            bool go = true;
            for (; more && go; more = w.next<NC>(a, lane)) {
                const int num_pages = (w.t_end + a.page_size - 1) >> a.page_shift;
                const int32_t *table = kv_table(a, w.req, w.begin);
                auto load_ids = [&](int p) { return p + lane < num_pages ? table[p + lane] : 0; };
                int batch = w.t_begin >> a.page_shift;  // page ids batch .. batch + 31 are in `ids`, one per lane
                int32_t ids = load_ids(batch), ids_next = load_ids(batch + 32);
                for (int t0 = w.t_begin; t0 < w.t_end && go; t0 += kTile) {
                    const int here = min(boxes, (w.t_end - t0 + box_rows - 1) >> box_shift);  // boxes with tokens
                    if ((t0 >> a.page_shift) >= batch + 32) {
                        batch += 32;
                        ids = ids_next;
                        ids_next = load_ids(batch + 32);
                    }
                    const int tb = t0 + (lane < boxes ? lane : 0) * box_rows;
                    int32_t id = __shfl_sync(0xffffffffu, ids, ((tb >> a.page_shift) - batch) & 31);
                    if (lane < here && (id < 0 || id >= a.num_pages)) {
                        report(a.status, DSA_ERR_BOUNDS);
                        id = 0;
                    }
                    const int y = (id * a.kv_heads + w.g) * 2 * a.page_size + (tb & (a.page_size - 1));
#pragma unroll 1
                    for (int v = 0; v < 2 && go; ++v) {  // K, then V
                        const uint32_t ring = v ? C::kV : C::kK, turn = issued / ring;
                        const uint32_t u = (v ? C::kK : 0) + issued - turn * ring;
                        if (!wait_mbar_warp(&empty[u], (turn & 1) ^ 1, abort)) {
                            gave_up(abort, a.status);
                            go = false;
                            break;
                        }
                        if (lane == 0) mbar_arrive_expect_tx(&full[u], here * box_rows * kDim);
                        __syncwarp();
                        if (lane < here)
                            tma_load_2d_hint(smem + u * kUnitBytes + lane * box_rows * kDim, &kv_map, &full[u], 0,
                                             y + v * a.page_size, policy);
                    }
                    ++issued;
                }
            }
            // (with many items only now, as in kv_attention_kernel; 4 x 8K: 14.6 us early, 12.9 so)
            if (!direct && !a.keep_parts) pdl_launch_dependents();
            if (*abort && lane == 0) {  // leave no copy in flight behind: the last tiles issued in either ring
                for (int v = 0; v < 2; ++v) {
                    const uint32_t ring = v ? C::kV : C::kK;
                    for (uint32_t i = issued > ring ? issued - ring : 0; i < issued; ++i) {
                        const long long t0 = clock64();
                        while (!mbar_try_wait(&full[(v ? C::kK : 0) + i % ring], (i / ring) & 1) &&
                               clock64() - t0 < kWaitTimeoutCycles) {
                        }
                    }
                }
            }
        } else if (warp == kQuery) {
            // ---- items, their columns and query images (rows hi 0 .. NC - 1, lo NC .. 2 NC - 1 of 128 bytes).
            // Neighbours of one row group and KV head share an image; the first is the softmax warps' work
            uint32_t count = 0, images = 1;  // items handed on, images begun
            bool go = true, fresh = false;
            if (more) named_bar_sync(2, 32 * (kSoftmax + 1));
            for (; more && go; more = w.next<NC>(a, lane)) {
                if (w.bad && w.part == 0 && lane == 0) report(a.status, DSA_ERR_BOUNDS);
                const uint32_t parity = count & 1;
                // a turn takes four columns, and the loads of the next turn run beside it: code that is not
                // used all the time comes from L2, at about 150 cycles for eight instructions
                uint4 v0, v1;
                if (fresh) load_query(a, w, lane >> 3, cols, hpg, lane, v0, v1);
                if (!wait_mbar_warp(&q_empty[parity], (count >> 1 & 1) ^ 1, abort)) {
                    gave_up(abort, a.status);
                    go = false;
                    break;
                }
                if (fresh) {
                    const uint32_t buf = images % C::kQBufs;
                    if (!wait_mbar_warp(&img_empty[buf], (images / C::kQBufs & 1) ^ 1, abort)) {
                        gave_up(abort, a.status);
                        go = false;
                        break;
                    }
#pragma unroll 1
                    for (int n = lane >> 3; n < NC; n += 4) {
                        const uint4 u0 = v0, u1 = v1;
                        load_query(a, w, n + 4 < NC ? n + 4 : cols, cols, hpg, lane, v0, v1);
                        convert_query<NC>(smem + C::OFF_Q + buf * C::kQBytes, cols_s + (images & 1), a, w, n, cols, hpg, u0,
                                          u1, lane);
                    }
                    ++images;
                }
                // the item after this one: a part more of the same row group and KV head?
                fresh = !(w.part + 1 < w.parts && w.start + kItemCost + ((w.t_end - w.t_begin + 127) >> 7) < w.end);
                Item *item = item_s + parity;
                if (lane < 8) item->ctx[lane] = w.my_ctx;
                if (lane == 0) {
                    item->live = 1;
                    item->t_begin = w.t_begin;
                    item->t_end = w.t_end;
                    item->ctx_min = w.ctx_min;
                    item->ctx_max = w.ctx;
                    item->cols = min(NC, cols - w.col0);
                    item->image_last = fresh;
                    item->part = w.part;
                    item->to_parts = w.parts > 1 || a.keep_parts;
                }
                fence_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&q_full[parity]);
                ++count;
            }
            if (go && wait_mbar_warp(&q_empty[count & 1], (count >> 1 & 1) ^ 1, abort) && lane == 0) {
                item_s[count & 1].live = 0;
                mbar_arrive(&q_full[count & 1]);
            }
        } else if (lane == 0) {
            // ---- the two MMA issuers, one thread each: an MMA's issue lasts as long as its passage through the
            // tensor core, so one thread for both products would set the pace
            const bool values = warp == kValues;
            // (formats: 0 e4m3, 1 e5m2)
            const uint32_t idesc = values ? make_idesc(kDim, C::kON, 0, 1, true, true)
                                           : make_idesc(kTile, C::kSN, 0, 0, false, false);
            const uint32_t idesc_turn = values ? make_idesc(kDim, NC, 0, 1, true, true) : idesc;  // (of one term)
            const uint32_t ring = values ? C::kV : C::kK, slot0 = values ? C::kK : 0;
            const uint32_t ua = smem_u32(smem);
            const uint64_t b0 = sdesc_sw128(smem_u32(smem + (values ? C::OFF_P : C::OFF_Q)), 16, 1024);
            const uint32_t step = values ? 256 : 2;
            uint32_t count = 0, p_phases = 0, o_phase = 1, image = 0;  // count: tiles
            bool ok = true;
            for (uint32_t n = 0; ok; ++n) {
                ok = wait_mbar(&q_full[n & 1], n >> 1 & 1, abort);
                if (!ok) break;
                const Item *item = item_s + (n & 1);
                const uint32_t buf = image % C::kQBufs;
                const uint64_t bd = values ? b0 : b0 + buf * (C::kQBytes / 16);
                if (item->live == 0) break;
                const int tiles = (item->t_end - item->t_begin + kTile - 1) / kTile;
                const bool image_last = item->image_last != 0;
                mbar_arrive(&q_empty[n & 1]);
                if (!values && image_last && tiles == 0) mma_commit(&img_empty[buf]);
                image += image_last;
                if (values && tiles > 0) {
                    ok = wait_mbar(o_empty, o_phase, abort);
                    o_phase ^= 1;
                }
                for (int i = 0; ok && i < tiles; ++i, ++count) {
                    const uint32_t turn = count / ring, slot = slot0 + count - turn * ring, sb = count % C::kSBufs;
                    const uint32_t pb = count % C::kPBufs;
                    ok = wait_mbar(&full[slot], turn & 1, abort);
                    // values: levels 0 accumulates in O^T.  Else one product for each context of the group, on a copy
                    // of O^T from which the softmax warps take its columns
                    int levels = 0;
                    bool apart = false;
                    while (ok) {
                        ok = values ? wait_mbar(&p_full[pb], p_phases >> pb & 1, abort)
                                    : wait_mbar(&s_empty[sb], ((count / C::kSBufs) & 1) ^ 1, abort);
                        p_phases ^= 1u << pb;
                        if (!ok) break;
                        tc_fence_after();
                        if (values && !apart) {
                            levels = *levels_s;
                            apart = levels > 0;
                        }
                        const uint32_t x = C::kApartInScores ? sb * C::kSN : C::kTmemX;
                        const uint32_t d = tmem + (!values ? sb * C::kSN : apart ? x : C::kTmemO);
                        const uint32_t add = values && i > 0 ? 1u : 0u;
                        const uint64_t ad = sdesc_sw128(ua + slot * kUnitBytes, 16, 1024);
                        // (of two accumulators in turn: the first and third terms, then the second ones)
                        const bool part = C::kApartTurns > 1 && apart, second = part && (levels & 1);
                        const uint32_t turns = !values ? C::kSTurns : second ? 1 : C::kOTurns;
                        const uint64_t bt = bd + (values ? pb * C::kPRow + (second ? NC / 16 : 0) : 0);
#pragma unroll 1
                        for (uint32_t m = 0; m < turns; ++m) {
                            const uint32_t id = part || m > 0 ? idesc_turn : idesc;
                            const uint64_t bm = bt + (m > 0 ? (values ? C::kP3Offset : NC * kDim / 16) : 0u);
                            const uint32_t far = values && m > 0 ? 4 : 2 * step;
#pragma unroll
                            for (uint32_t j = 0; j < 4; ++j)
                                mma_f8(d, ad + j * step, bm + (j & 1) * step + (j >> 1) * far, id, m + j > 0 ? 1u : add);
                        }
                        --levels;
                        if (levels <= 0) mma_commit(&empty[slot]);
                        mma_commit(values ? &pv_done[pb] : &s_full[sb]);
                        if (levels <= 0) break;
                    }
                    if (!values && ok && image_last && i == tiles - 1) mma_commit(&img_empty[buf]);
                }
            }
            if (!ok) gave_up(abort, a.status);
            if (*abort) {  // leave no MMA in flight behind
                mma_commit(drained);
                const long long t0 = clock64();
                while (!mbar_try_wait(drained, 0) && clock64() - t0 < kWaitTimeoutCycles) {
                }
            }
        }
        __syncwarp();
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::kSoftmaxRegs));
        // ---- softmax: thread = token (TMEM lane) of a tile, then dim of the output.  A wait that gives up makes
        // its warp `dead`.  Every meeting whose first round is true has a second one that asks for dead warps,
        // after which all leave: so no warp waits for one that has gone
        const int self = (warp & 3) * 32 + lane;
        const int mine = (warp >> 2) * kMine;   // this warpgroup's first column
        const uint32_t quad = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + mine;
        float *max_s = reinterpret_cast<float *>(smem + C::OFF_MAX) + 4 * mine;  // [4][kMine], as the sums
        float *nbase = reinterpret_cast<float *>(smem + C::OFF_BASE) + warp * kMine;
        float *fac = reinterpret_cast<float *>(smem + C::OFF_FAC) + warp * kMine;
        float *move = reinterpret_cast<float *>(smem + C::OFF_MOVE) + warp * kMine;
        uint32_t s_count = 0;                   // tiles
        uint32_t pv_open = 0, pv_phases = 0;    // a bit per buffer of P: a product is out whose end has not been seen
        if (more) {  // the first item's columns, four a warp and turn
#pragma unroll 1
            for (int n = 4 * warp + (lane >> 3); n < NC; n += 4 * kSoftmax) {
                uint4 v0, v1;
                load_query(a, w, n, cols, hpg, lane, v0, v1);
                convert_query<NC>(smem + C::OFF_Q, cols_s, a, w, n, cols, hpg, v0, v1, lane);
            }
            fence_async_smem();
            asm volatile("bar.arrive 2, %0;" ::"n"(32 * (kSoftmax + 1)) : "memory");
        }
        bool dead = false;
        uint32_t image = 0;
        auto pv_wait = [&](uint32_t b) {
            if (!(pv_open >> b & 1)) return;
            dead |= !wait_mbar_warp(&pv_done[b], pv_phases >> b & 1, abort);
            pv_phases ^= 1u << b;
            pv_open &= ~(1u << b);
            tc_fence_after();
        };
        auto pv_wait_all = [&]() {
#pragma unroll
            for (uint32_t b = 0; b < C::kPBufs; ++b) pv_wait(b);
        };
        auto meet_any = [](bool p) { return meet_any_of<32 * kSoftmax>(p); };
        auto someone_dead = [&]() { return meet_any(dead) && meet_any(dead); };
        for (uint32_t item_n = 0;; ++item_n) {
            const uint32_t parity = item_n & 1;
            dead |= !wait_mbar_warp(&q_full[parity], item_n >> 1 & 1, abort);
            const Item *item = item_s + parity;
            if (dead || item->live == 0) {
                someone_dead();
                break;
            }
            const Columns<NC> *cs = cols_s + (image & 1);
            image += item->image_last != 0;
            const int t_begin = item->t_begin, t_end = item->t_end, ctx_min = item->ctx_min, ctx_max = item->ctx_max;
            const int ncols = item->cols, part = item->part, to_parts = item->to_parts;
            const int tiles = (t_end - t_begin + kTile - 1) / kTile;

            float l[kMine];  // a thread's sums of weights, unless they are in TMEM
#pragma unroll
            for (int n = 0; n < kMine; ++n) l[n] = 0.f;
            if constexpr (C::kSumsInTmem) {
                uint32_t zeros[16];
#pragma unroll
                for (int j = 0; j < 16; ++j) zeros[j] = 0u;
#pragma unroll
                for (int c = 0; c < kMine; c += 16) tmem_st16(quad + C::kTmemL + c, zeros);
                tmem_st_wait();
            }
#pragma unroll 1
            for (int n = lane; n < kMine; n += 32) nbase[n] = 0.f;
            __syncwarp();
            bool leave = false;
            for (int i = 0; i < tiles; ++i, ++s_count) {
                const int t0 = t_begin + i * kTile, t = t0 + self;
                const uint32_t sb = s_count % C::kSBufs, pb = s_count % C::kPBufs;
                const uint32_t v_turn = s_count / C::kV, vslot = C::kK + s_count - v_turn * C::kV;
                uint4 *vrow = reinterpret_cast<uint4 *>(smem + vslot * kUnitBytes + self * kDim);
                dead |= !wait_mbar_warp(&s_full[sb], (s_count / C::kSBufs) & 1, abort);
                tc_fence_after();
                const bool edge = t0 + kTile > ctx_min;  // some column does not see all of the tile

                // scores of this token in log2 units against their bases
                auto scores = [&](float (&x)[kMine]) {
                    uint32_t h[kMine];
                    if constexpr (C::kSN > NC) {
                        uint32_t g[16];
                        tmem_ld16(quad + sb * C::kSN, h);
                        tmem_ld16(quad + sb * C::kSN + NC, g);
                        tmem_ld_wait();
                        reg_fence(h);
                        reg_fence(g);
                        add16(h, g);
                    } else {
                        tmem_ld32(quad + sb * C::kSN, h);
                        tmem_ld_wait();
                        reg_fence(h);
                    }
#pragma unroll
                    for (int j = 0; j < kMine; j += 4) {
                        const float4 sc = *reinterpret_cast<const float4 *>(cs->scale + mine + j);
                        const float4 nb = *reinterpret_cast<const float4 *>(nbase + j);
                        const float2 p = __ffma2_rn(make_float2(__uint_as_float(h[j]), __uint_as_float(h[j + 1])),
                                                    make_float2(sc.x, sc.y), make_float2(nb.x, nb.y));
                        const float2 q = __ffma2_rn(make_float2(__uint_as_float(h[j + 2]), __uint_as_float(h[j + 3])),
                                                    make_float2(sc.z, sc.w), make_float2(nb.z, nb.w));
                        x[j] = p.x;
                        x[j + 1] = p.y;
                        x[j + 2] = q.x;
                        x[j + 3] = q.y;
                    }
                    if (edge) {
#pragma unroll
                        for (int j = 0; j < kMine; j += 4) {
                            const int4 n = *reinterpret_cast<const int4 *>(cs->ctx + mine + j);
                            if (t >= n.x) x[j] = -INFINITY;
                            if (t >= n.y) x[j + 1] = -INFINITY;
                            if (t >= n.z) x[j + 2] = -INFINITY;
                            if (t >= n.w) x[j + 3] = -INFINITY;
                        }
                    }
                };
                float x[kMine];
                scores(x);
                const bool keep = C::kSBufs > 1 || edge;  // an only buffer goes back at once, unless it is of use once more
                if (!keep) {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&s_empty[sb]);
                }
                float top = -INFINITY;
#pragma unroll
                for (int j = 0; j < kMine; j += 2) top = fmaxf(top, fmaxf(x[j], x[j + 1]));
                // the first tile sets the bases; later, when a score no longer fits, all columns' are raised to where a
                // move leaves them, so that the next one is further off
                if (i == 0 || meet_any(top > kTop || dead)) {
                    max_columns<kMine>(x, max_s + (warp & 3) * kMine, lane);
                    if (i == 0 ? someone_dead() : meet_any(dead)) {
                        leave = true;
                        break;
                    }
                    pv_wait_all();  // O^T at rest
#pragma unroll 1
                    for (int n = lane; n < kMine; n += 32) {
                        const float m = fmaxf(fmaxf(max_s[n], max_s[kMine + n]),
                                              fmaxf(max_s[2 * kMine + n], max_s[3 * kMine + n]));
                        const float by = m > (i == 0 ? -INFINITY : kBias) ? kBias - m : 0.f;
                        move[n] = by;
                        fac[n] = ex2(by);
                        nbase[n] += by;
                    }
                    __syncwarp();
#pragma unroll
                    for (int j = 0; j < kMine; j += 4) {
                        const float4 by = *reinterpret_cast<const float4 *>(move + j);
                        x[j] += by.x;
                        x[j + 1] += by.y;
                        x[j + 2] += by.z;
                        x[j + 3] += by.w;
                    }
                    if (i > 0) {
                        if (!C::kSumsInTmem) {
#pragma unroll
                            for (int n = 0; n < kMine; ++n) l[n] *= fac[n];
                        }
                        // O^T and the sums in TMEM lie NC columns apart
#pragma unroll 1
                        for (uint32_t at = C::kTmemO; at < C::kTmemL + (C::kSumsInTmem ? NC : 0); at += NC) {
#pragma unroll 1
                            for (int c = 0; c < kMine; c += 16) {
                                uint32_t h[16];
                                tmem_ld16(quad + at + c, h);
                                tmem_ld_wait();
                                reg_fence(h);
#pragma unroll
                                for (int j = 0; j < 16; ++j) h[j] = __float_as_uint(__uint_as_float(h[j]) * fac[c + j]);
                                tmem_st16(quad + at + c, h);
                            }
                        }
                        tmem_st_wait();
                    }
                }
                pv_wait(pb);  // this buffer of P is free

                // weights, 16 columns at a time
#pragma unroll
                for (int c = 0; c < kMine; c += 16) {
                    if constexpr (C::kSumsInTmem) {
#pragma unroll
                        for (int j0 = 0; j0 < 16; j0 += 8) {  // eight at a time, for want of registers
                            uint32_t sums[8];
                            tmem_ld8(quad + C::kTmemL + c + j0, sums);
#pragma unroll
                            for (int j = j0; j < j0 + 8; ++j) x[c + j] = ex2(x[c + j]);
                            tmem_ld_wait();
                            reg_fence(sums);
#pragma unroll
                            for (int j = 0; j < 8; j += 2)
                                add_pair(sums[j], sums[j + 1], x[c + j0 + j], x[c + j0 + j + 1]);
                            tmem_st8(quad + C::kTmemL + c + j0, sums);
                        }
                    } else {
#pragma unroll
                        for (int j = 0; j < 16; ++j) x[c + j] = ex2(x[c + j]);
#pragma unroll
                        for (int j = 0; j < 16; j += 2) {
                            const float2 s = __fadd2_rn(make_float2(l[c + j], l[c + j + 1]), make_float2(x[c + j], x[c + j + 1]));
                            l[c + j] = s.x;
                            l[c + j + 1] = s.y;
                        }
                    }
                    uint32_t t1[4], t2[4], t3[4];
#pragma unroll
                    for (int j = 0; j < 16; j += 4)
                        weight_terms(pack_f16(x[c + j], x[c + j + 1]), pack_f16(x[c + j + 2], x[c + j + 3]), t1[j / 4],
                                     t2[j / 4], t3[j / 4]);
                    const int at = C::kPRow * pb + (mine + c) / 16;
                    uint8_t *p_s = smem + C::OFF_P;
                    *reinterpret_cast<uint4 *>(p_s + sw128(self, at)) = make_uint4(t1[0], t1[1], t1[2], t1[3]);
                    *reinterpret_cast<uint4 *>(p_s + sw128(self, at + NC / 16)) = make_uint4(t2[0], t2[1], t2[2], t2[3]);
                    const uint32_t third = NC < 64 ? sw128(self, at + 2 * NC / 16)
                                                   : kTile * 128 + sw128(self & 63, (self >> 6) * 4 + (mine + c) / 16);
                    *reinterpret_cast<uint4 *>(p_s + third) = make_uint4(t3[0], t3[1], t3[2], t3[3]);
                }
                if (C::kSumsInTmem) tmem_st_wait();
                auto hand_over = [&]() {
                    fence_async_smem();
                    tc_fence_before();
                    __syncwarp();
                };
                bool apart = false;
                if (edge) {
                    dead |= !wait_mbar_warp(&full[vslot], v_turn & 1, abort);
                    if (a.group > 1) {  // is a V code that only some rows see NaN?
                        bool nan = false;
                        if (t >= ctx_min && t < ctx_max) {
#pragma unroll
                            for (int y = 0; y < 8; ++y) {
                                const uint4 v = vrow[y];
                                nan |= any_nan4(v.x) || any_nan4(v.y) || any_nan4(v.z) || any_nan4(v.w);
                            }
                        }
                        apart = meet_any(nan || dead);
                        if (apart && meet_any(dead)) {
                            leave = true;
                            break;
                        }
                    }
                    if (mine == 0 && t >= ctx_max) {  // no row sees it: whatever the slot or the stage holds
#pragma unroll
                        for (int y = 0; y < 8; ++y) vrow[y] = make_uint4(0u, 0u, 0u, 0u);
                    }
                }
                if (!apart) {
                    hand_over();
                    if (lane == 0) {
                        if (keep) mbar_arrive(&s_empty[sb]);
                        mbar_arrive(&p_full[pb]);
                    }
                    pv_open |= 1u << pb;
                    continue;
                }
                // 0 x NaN must not reach the rows that do not see it.  One product per context of the group,
                // longest first, with V's tokens past it zeroed, on a copy of O^T (so a column's bits are those of the
                // one product for all); of each only the columns of that context are taken over.
                pv_wait_all();  // O^T at rest
                int levels = 0;
                for (int prev = INT32_MAX;; ++levels) {
                    int next = -1;
                    for (int r = 0; r < a.group; ++r)
                        if (item->ctx[r] < prev) next = max(next, item->ctx[r]);
                    if (next < 0) break;
                    prev = next;
                }
                levels *= C::kApartTurns;
                if (threadIdx.x == 0) *levels_s = levels;
                const uint32_t xo = quad + (C::kApartInScores ? sb * C::kSN : C::kTmemX);
                for (int v = 0, cur = INT32_MAX; v < levels; ++v) {
                    const uint32_t of = quad + C::kTmemO + v % C::kApartTurns * C::kXN;
                    if (v % C::kApartTurns == 0) {
                        int next = -1;
                        for (int r = 0; r < a.group; ++r)
                            if (item->ctx[r] < cur) next = max(next, item->ctx[r]);
                        cur = next;
                        if (mine == 0 && t >= cur) {
#pragma unroll
                            for (int y = 0; y < 8; ++y) vrow[y] = make_uint4(0u, 0u, 0u, 0u);
                        }
                    }
                    if (i > 0) {
#pragma unroll 1
                        for (int c = 0; c < kMine; c += 16) {
#pragma unroll 1
                            for (int y = c; y < C::kXN; y += NC) {
                                uint32_t g[16];
                                tmem_ld16(of + y, g);
                                tmem_ld_wait();
                                reg_fence(g);
                                tmem_st16(xo + y, g);
                            }
                        }
                        tmem_st_wait();
                    }
                    hand_over();
                    if (lane == 0) mbar_arrive(&p_full[pb]);
                    pv_open |= 1u << pb;
                    pv_wait(pb);
#pragma unroll 1
                    for (int c = 0; c < kMine; c += 16) {
#pragma unroll 1
                        for (int y = c; y < C::kXN; y += NC) {
                            uint32_t h[16], g[16];
                            tmem_ld16(xo + y, h);
                            tmem_ld16(of + y, g);
                            tmem_ld_wait();
                            reg_fence(h);
                            reg_fence(g);
#pragma unroll
                            for (int j = 0; j < 16; ++j)
                                if (cs->ctx[mine + c + j] == cur) g[j] = h[j];
                            tmem_st16(of + y, g);
                        }
                    }
                    tmem_st_wait();
                }
                tc_fence_before();
                __syncwarp();
                if (threadIdx.x == 0) *levels_s = 0;
                if (keep && lane == 0) mbar_arrive(&s_empty[sb]);
            }
            if (leave) break;

            // ---- the item's sums and output
            float *sums = sum_s + parity * 4 * NC + 4 * mine;
            if (C::kSumsInTmem) {
#pragma unroll
                for (int c = 0; c < kMine; c += 16) {
                    uint32_t h[16];
                    tmem_ld16(quad + C::kTmemL + c, h);
                    tmem_ld_wait();
                    reg_fence(h);
#pragma unroll
                    for (int j = 0; j < 16; ++j) l[c + j] = __uint_as_float(h[j]);
                }
            }
            reduce_columns<kMine>(l, sums + (warp & 3) * kMine, lane);
            if (someone_dead()) break;
            // a column's factor where the part is the whole: 1 / its sum (0 without any weight)
#pragma unroll 1
            for (int n = lane; n < kMine; n += 32) {
                const float total = sums[n] + sums[kMine + n] + sums[2 * kMine + n] + sums[3 * kMine + n];
                fac[n] = total == 0.f ? 0.f : a.v_scale / total;
                if ((warp & 3) == 0 && mine + n < ncols) {
                    const float b = -nbase[n];
                    const int at = cs->at[mine + n];
                    if (to_parts)
                        a.part_ml[static_cast<int64_t>(at) * a.parts_bound + part] = make_float2(part_base(b, total), total);
                    else if (a.lse != nullptr)
                        a.lse[at] = total == 0.f ? -INFINITY : (b + log2f(total)) * 0.6931471805599453f;
                }
            }
            __syncwarp();
            pv_wait_all();
            // thread = dim: a warp's lanes write 32 dims of a column in a row
#pragma unroll 1
            for (int c = 0; c < min(ncols - mine, kMine); c += 16) {
                uint32_t h[16];
                tmem_ld16(quad + C::kTmemO + c, h);
                tmem_ld_wait();
                reg_fence(h);
#pragma unroll
                for (int y = NC; y < C::kON; y += NC) {
                    uint32_t g[16];
                    tmem_ld16(quad + C::kTmemO + y + c, g);
                    tmem_ld_wait();
                    reg_fence(g);
                    add16(h, g);
                }
                const int here = ncols - mine - c;
                if (to_parts) {  // (a part without tiles, the only one of its group, is not looked at)
                    float *dst = a.part_o + part * kDim + self;
                    const int64_t row = static_cast<int64_t>(a.parts_bound) * kDim;
#pragma unroll
                    for (int j = 0; j < 16; j += 4) {
                        const int4 at = *reinterpret_cast<const int4 *>(cs->at + mine + c + j);
                        if (j < here) dst[at.x * row] = __uint_as_float(h[j]);
                        if (j + 1 < here) dst[at.y * row] = __uint_as_float(h[j + 1]);
                        if (j + 2 < here) dst[at.z * row] = __uint_as_float(h[j + 2]);
                        if (j + 3 < here) dst[at.w * row] = __uint_as_float(h[j + 3]);
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        if (j >= here) break;
                        const float f = fac[c + j], o = f == 0.f ? 0.f : __uint_as_float(h[j]) * f;
                        a.out[static_cast<int64_t>(cs->at[mine + c + j]) * kDim + self] =
                            __bfloat16_as_ushort(__float2bfloat16_rn(o));
                    }
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                if (tiles > 0) mbar_arrive(o_empty);
                mbar_arrive(&q_empty[parity]);
            }
        }
        if (dead) gave_up(abort, a.status);
    }
    __syncthreads();
    if (warp == kScores) {
        tc_fence_after();
        tmem_dealloc(tmem, C::kTmemCols);
    }
}

template <int NC>
cudaError_t launch_columns(KvAttnArgs &a, int cols, cudaStream_t s) {
    a.col_blocks = (cols + NC - 1) / NC;
    const int64_t items = static_cast<int64_t>(a.num_rows / a.group) * a.kv_heads * a.col_blocks * a.parts_bound;
    if (items > 0x7fffffff) return cudaErrorInvalidConfiguration;
    a.items = static_cast<uint32_t>(items);
    static std::atomic<uint64_t> configured{0};
    cudaError_t e = raise_smem_limit(kv_attention_fp8_kernel<NC>, Cfg<NC>::kSmemBytes, configured);
    if (e != cudaSuccess) return e;
    // the register split waits forever in a CTA launched with fewer
    static std::atomic<int> regs{0};
    if (regs.load() == 0) {
        cudaFuncAttributes fa;
        e = cudaFuncGetAttributes(&fa, kv_attention_fp8_kernel<NC>);
        if (e != cudaSuccess) return e;
        regs.store(fa.numRegs);
    }
    if (regs.load() < Cfg<NC>::kLaunchRegs) return cudaErrorInvalidConfiguration;
    CUtensorMap map;
    if (!encode_kv_rows_map(&map, a.pool, a.pool_rows, kDim, a.page_size)) return cudaErrorInvalidValue;
    const uint32_t ctas = persistent_ctas(a);
    if (ctas == 0) return cudaErrorInvalidDevice;
    return launch_pdl(kv_attention_fp8_kernel<NC>, dim3(ctas), dim3(Cfg<NC>::kThreads), Cfg<NC>::kSmemBytes, s, map, a);
}

}  // namespace

cudaError_t launch_kv_attention_fp8(KvAttnArgs &a, cudaStream_t s) {
    const int cols = a.group * (a.num_heads / a.kv_heads);
    if (cols <= 16) return launch_columns<16>(a, cols, s);
    if (cols <= 32) return launch_columns<32>(a, cols, s);
    return launch_columns<64>(a, cols, s);
}

}  // namespace dsa
