// kv_attention_shared.cu -- attention of a batch whose rows share prefixes (dsa_kv_attention_shared).
//
//   out[r, h, :] = sum_t softmax_t(sm_scale <q[r,h,:], K_g,t>) V_g,t   over t < row_ctx[r],
//
// where the tokens before a segment's S are the same for all of its rows.  The sum is split at S: the shared tokens are
// read once for all rows of the segment (kv_shared_kernel), each row reads the others by itself (kv_attention.cu, from
// an offset into its table, on SMs of its own), and kv_join_kernel adds the parts up by log-sum-exp.  kv_segments_kernel
// works out S, a multiple of 128, and who does what.  S is at most what every row of the segment that sees any token
// sees, so no score of a shared token is ever masked, whatever its V holds.
//
// A token of a KV head is 4 D bytes in bf16 (2 D in e4m3) and serves N = rows x query heads per KV head columns at
// 4 D FLOP each: from N = 300 in bf16 (150 in e4m3) on the products take longer than the bytes.  So the columns go on
// M, the tensor core's 128 rows, twice:
//
//   S[128 columns x 128 tokens] = Q K^T     Q and K from shared memory, S in TMEM
//   P = 2^(S - b)                           a thread a column: it reads its row of S, keeps its base and sum in registers
//                                           and puts P over S in TMEM, in 16 bits
//   O[128 columns x D] += P V               P from TMEM, V from shared memory, O in TMEM for the whole item
//
// A CTA (one an SM: 512 TMEM columns, 182 to 231 KB) has two such chains, each with a warpgroup for its softmax and a warp
// that issues its products, so that one's products run beside the other's exponentials.  An item of more than 128 columns
// has 128 for each chain, and every tile of K and V serves both; one of fewer has the same columns in both, which then
// take every other tile.  K and V come by TMA, a warp and a ring each.
//
// What bounds it (4 KV heads of 128, in a graph): many rows, the chain of a tile: 1,024 cycles of MMA, 830 of
// exponentials, 500 to 600 of waits between them, so that two chains take 2,350 (bf16) to 2,450 (FP8) cycles a tile where
// the tensor core needs 2,048.  256 rows of 64K, 16 query heads each: 550 GFLOP in 351 us (1.57 PFLOP/s, 0.82 of cuBLAS's
// burst), 128 SMs at the shared tokens for 325 of them.  64 rows of 64K and 8, bf16: 69 us for 36 of products.  Few rows,
// bytes: 4 rows of 128K, bf16 65 us, 268 MB.  Below that the latencies of four kernels: checks 6, a shared item's start
// (7,000 cycles to its first weights) and output (6,300: 128 KB at what an SM writes) 7, join 5 us.  Head_dim 64 has
// half the products and as many exponentials: 256 rows of 32K, 16 query heads each, FP8 168 us and bf16 199 against 72 of
// products.
//
// Precision.  bf16 pool: products are exact, P is rounded to bf16 (2^-8 of itself; kv_attention.cu's second term would
// make the second product, half of all, twice as long).  FP8 pool: q as two e4m3 terms against K's codes as they
// are, V's codes exactly as fp16 (a third warpgroup converts them) and P rounded to fp16 (2^-11, in steps of 2^-24 with
// the largest at 2^7 or more).
#include "kv_attention_common.cuh"
#include "mla_fp8_common.cuh"

namespace dsa {

namespace {

using namespace kv;
using fp8mla::split_pair;

constexpr int kTile = 128;       // tokens of a tile, and columns of a chain
constexpr int kSharedCtas = 152;  // an SM each; a constant, so that the split does not go by the device

// A segment's work.
struct alignas(16) KvSharedSeg {
    int32_t row0, rows;
    int32_t tiles;          // of its shared tokens
    int32_t req;            // whose block table lists them
    int32_t parts, blocks;  // an item is a (KV head, block of 256 columns, part of the tiles)
    int32_t entries;        // outputs of a (row, head): one a part, or two where chains share the columns
    int32_t cost;           // of an item, in tiles of one chain
    int64_t entry0, cost0;  // before the segment's
};
static_assert(sizeof(KvSharedSeg) == 48, "segment layout");

// Where a CTA begins, and the cost at which its share of all ends.
struct alignas(16) KvSharedCta {
    int32_t seg, item;  // seg -1: nothing to do
    int64_t end;
};

struct KvSharedArgs {
    KvAttnArgs a;                 // row_ctx: what a row reads itself
    const int32_t *row_ctx;       // the call's
    const int32_t *first_row, *shared_ctx;
    int32_t num_segments;
    int64_t least_saved;          // bytes, in a segment
    int32_t *own_ctx, *row_begin, *row_seg;  // [R]; row_seg: -1 where nothing is shared
    KvSharedSeg *seg;             // [num_segments]
    KvSharedCta *cta;             // [kSharedCtas]
    float *so;                    // [entry][H][D]
    float2 *sml;                  // [entry][H]
    int32_t *own_sms;             // SMs that the rows' own tokens take while the others read shared ones
    bool beside;                  // whether they do
    float own_tile, own_item;     // what a tile of them and an item cost an SM, in tiles of a chain
    uint8_t *q_terms;             // FP8: [R][H][2][D] e4m3, hi and lo terms of the queries times 2^e
    float *q_factor;              // [R][H] 2^-e (NaN: not only numbers in the query)
};

// (an early_read)
__device__ __forceinline__ KvSharedSeg read_segment(const KvSharedSeg *p) {
    union {
        int4 words[3];
        KvSharedSeg seg;
    } u;
#pragma unroll
    for (int i = 0; i < 3; ++i) u.words[i] = early_read(reinterpret_cast<const int4 *>(p) + i);
    return u.seg;
}

// Rows' own tokens in parts of 2^10 at least where a segment has so many (row group, KV head): 32 rows of 4 KV heads and 32K
// tokens, with 100 to 4,096 of their own: 50.7 us, with 2^9 53.6, with 2^8 57.7; 256 rows of 64K 354 and with 2^8 436; but
// four segments of 4 groups of 4 rows 60.5 and 54.8.  us with 2^10 / 2^8 everywhere, 16 query heads a KV head:
//   (row group, KV head) of a segment     16         32         48         64         80         96         128        256
//   one segment of 32K, FP8             31.4/29.7  36.3/31.7  40.7/36.6  38.1/38.3  47.3/50.0  47.2/52.6  49.3/55.8  86/103
//                       bf16            31.4/28.8  36.6/34.4  39.0/40.3  42.7/40.0  49.5/50.8  52.0/54.4  56.1/59.9  89/105
//   four segments of 16K, FP8           38.2/41.7  50.6/59.1             63.5/78.8             109/141    114/145
//                       bf16            51.8/57.2  64.7/73.3             95/110                125/144    171/205
// So for rows one by one the rule turns late (the parts pay from 80, beside other segments from 16); for rows in groups, 16
// to a segment, they cost.
constexpr int32_t kManyGroups = 128, kManyPartMin = 10;
constexpr int32_t kItemTiles = 12;  // what an item costs beside its tiles
constexpr int32_t kMinTiles = 4;    // of a part

// Bytes that sharing has to save (those that the other rows of a segment would read) to make up for two launches more and
// another chain of latencies.  A call whose shapes leave less is dsa_kv_attention's (with dev_status, one launch more for the
// segments' checks: 10.3 us for 8.8); in one that is not, where half of that is spent already, a segment has to save half,
// and of several each its share.  The shapes are the rows and max_ctx, all that the host knows: with a bound far above the
// contexts a small batch goes through all four kernels with little or nothing shared (4 rows of 2K, bf16, max_ctx 131,072:
// 18.0 us, by dsa_kv_attention 10.6; 8 rows of 8K, FP8 24.5 and 20.6, bf16 22.8 and 24.1).
// us in a graph, 1 to 200 tokens of their own, each row by itself / in a call that shares nothing / shared:
//                       FP8, 4 heads of 128      bf16, 4 heads of 128     bf16, 3 heads of 64
//   8 rows of 8K         56 MB  21 / 29 / 26     112 MB  20 / 28 / 24      42 MB  12 / 19 / 19
//   16 rows of 8K       120 MB  30 / 38 / 27     240 MB  28 / 36 / 24      90 MB  18 / 25 / 20
//   64 rows of 1K        63 MB  30 / 34 / 28     126 MB  25 / 30 / 24      47 MB  14 / 21 / 21
//   64 rows of 2K       126 MB  42 / 47 / 30     252 MB  35 / 42 / 24      95 MB  19 / 25 / 22
//   4 rows of 32K        96 MB  26 / 34 / 32     192 MB  27 / 35 / 29      72 MB  16 / 24 / 21
int64_t shared_least_bytes(const KvAttnArgs &a) {
    const int64_t mb = a.fp8 ? 100 : 160;
    return (a.head_dim == 64 ? mb * 2 / 3 : mb) << 20;
}

__host__ __device__ __forceinline__ int64_t token_bytes(const KvAttnArgs &a) {
    return 2ll * a.kv_heads * a.head_dim * (a.fp8 ? 1 : 2);
}

// The most parts of a segment with so many items a part: an item a CTA where that is possible, else few enough that their
// outputs stay small beside the products, and enough to fill the last round of CTAs.
__host__ __device__ __forceinline__ int32_t shared_parts_cap(int32_t units) {
    return units <= kSharedCtas / 8 ? kSharedCtas / units : units <= kSharedCtas ? 8 : units <= 4 * kSharedCtas ? 4 : 2;
}

// ------------------------------------------------------------------ who reads what

// One CTA.  Its time is that of a chain of dependent reads, so what it goes through again stays in shared memory while it
// fits.  A warp takes a segment, so from 8 on they follow one another: us by itself, cold, for 1 / 16 / 64 / 128 segments
// 8 / 10 / 20 / 33.  Of 128 pairs of rows (FP8, 4 heads of 128, 8 query heads each) sharing 2,048 tokens takes 144 us and
// each by itself 139, of 4,096 tokens 184 and 234.
constexpr int kSegThreads = 256, kSegRows = 8192, kSegSegs = 64;

// put(segment, first row, rows, shared tokens) of every segment, of no rows where it cannot be, which is reported.  All
// threads of the CTA.
template <typename Put>
__device__ __forceinline__ void check_segments(const KvSharedArgs &s, int32_t *tops, const Put &put) {
    const KvAttnArgs &a = s.a;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // a segment begins at or behind every bound before it
    const int per = (s.num_segments + kSegThreads) / kSegThreads;
    const int lo = min(s.num_segments + 1, static_cast<int>(threadIdx.x) * per);
    const int hi = min(s.num_segments + 1, lo + per);
    int32_t top = INT32_MIN;
    for (int i = lo; i < hi; ++i) top = max(top, s.first_row[i]);
    int32_t upto = top;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int32_t u = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto = max(upto, u);
    }
    if (lane == 31) tops[warp] = upto;
    top = __shfl_up_sync(0xffffffffu, upto, 1);
    if (lane == 0) top = INT32_MIN;
    __syncthreads();
    for (int t = 0; t < warp; ++t) top = max(top, tops[t]);
    for (int i = lo; i < min(hi, s.num_segments); ++i) {
        const int32_t first = s.first_row[i], end = s.first_row[i + 1], shared = s.shared_ctx[i];
        const bool bad = first < 0 || first < top || end < first || end > a.num_rows || first % a.group != 0 ||
                         end % a.group != 0 || shared < 0;
        if (bad) report(a.status, DSA_ERR_BOUNDS);
        put(i, bad ? 0 : first, bad ? 0 : end - first, bad ? 0 : shared);
        top = max(top, first);
    }
}

// The queries over an FP8 pool as two e4m3 terms, times 2^e which brings a query's largest value to (224, 448], for all
// parts of its columns at once: by CTAs beside the one that works out the segments, in the time that it takes (each part
// for itself took 6,600 cycles before its first scores, a copy of the terms takes 2,300).  D / 16 lanes take a query.
template <int D>
__device__ __forceinline__ void split_queries(const KvSharedArgs &s, int cta, int ctas) {
    constexpr int kLanes = D / 16, kAt = 32 / kLanes;
    const KvAttnArgs &a = s.a;
    const int lane = threadIdx.x & 31, unit = lane % kLanes;
    const int64_t pairs = static_cast<int64_t>(a.num_rows) * a.num_heads;
    const int64_t warps = static_cast<int64_t>(ctas) * (kSegThreads / 32);
    for (int64_t p0 = (cta * (kSegThreads / 32) + (threadIdx.x >> 5)) * kAt; p0 < pairs; p0 += warps * kAt) {
        const int64_t p = p0 + lane / kLanes;
        uint4 v0 = make_uint4(0u, 0u, 0u, 0u), v1 = v0;
        if (p < pairs) {
            const int64_t row = p / a.num_heads;
            const uint4 *q = reinterpret_cast<const uint4 *>(a.q + row * a.q_stride + (p - row * a.num_heads) * D) + 2 * unit;
            v0 = q[0];
            v1 = q[1];
        }
        const uint32_t h[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
        uint32_t top = 0;  // by the bits: an infinity or a NaN is above every number
#pragma unroll
        for (int y = 0; y < 8; ++y) top = max(top, max(h[y] << 16 & 0x7fff0000u, h[y] & 0x7fff0000u));
#pragma unroll
        for (int y = 1; y < kLanes; y <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, y));
        const bool finite = top < 0x7f800000u;
        int e = 0;
        if (top > 0 && finite) {
            e = 135 - static_cast<int>(top >> 23) - ((top & 0x7fffffu) > 0x600000u ? 1 : 0);
            e = max(-120, min(120, e));
        }
        const float up = __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int y = 0; y < 4; ++y) {
            const uint2 x = split_pair(bf16_lo(h[2 * y]) * up, bf16_hi(h[2 * y]) * up);
            const uint2 z = split_pair(bf16_lo(h[2 * y + 1]) * up, bf16_hi(h[2 * y + 1]) * up);
            hi[y] = x.x | (z.x << 16);
            lo[y] = x.y | (z.y << 16);
        }
        if (p >= pairs) continue;
        uint4 *to = reinterpret_cast<uint4 *>(s.q_terms + p * (2 * D)) + unit;
        to[0] = make_uint4(hi[0], hi[1], hi[2], hi[3]);
        to[D / 16] = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        if (unit == 0)
            s.q_factor[p] = finite ? __uint_as_float(static_cast<uint32_t>(127 - e) << 23) : __uint_as_float(0x7fc00000u);
    }
}

// What a row group's own tokens cost, for one KV head and block of columns.
__device__ __forceinline__ float own_cost(const KvSharedArgs &s, int32_t ctx, int32_t part_min) {
    if (ctx <= 0) return 0.f;
    const int32_t parts = kv_parts(ctx, kv_part_shift(ctx, kv_parts_shift(s.a.kv_heads), part_min));
    return static_cast<float>((ctx + kTile - 1) / kTile) * s.own_tile + static_cast<float>(parts) * s.own_item;
}

template <typename T>
__device__ __forceinline__ T warp_sum(T x) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

// The rows' own tokens wait for memory most of the time and the shared ones for the tensor core, and an SM has room for
// one of the two kernels.  So the own ones get some SMs (KvAttnArgs.own_sms) and the shared ones the others, so many that
// both end together, or all SMs one after the other where that is as good.  us, one after the other / beside: 32 rows of
// 32K and 100 to 4,096 59.6 / 49.3, verify rows of 16 requests 60.4 / 52.4, 256 rows of 64K 367 / 351, 64 rows of 64K
// bf16 71 / 69, 45 ragged rows of head_dim 64 24.9 / 23.0.
constexpr int kFewestSms = 8, kMostSms = kSharedCtas - 4;

__device__ __forceinline__ float rounds_of(float items, float sms) { return ceilf(__fdiv_rn(items, sms)); }

// CTA 0: the segments; the others, over an FP8 pool: the queries' terms.
__global__ void __launch_bounds__(kSegThreads, 1) kv_segments_kernel(const __grid_constant__ KvSharedArgs s) {
    const KvAttnArgs &a = s.a;
    __shared__ int32_t tops[kSegThreads / 32];
    __shared__ unsigned long long own_s;  // what the rows' own tokens cost
    __shared__ int sms_s;                 // for the shared ones
    __shared__ int32_t ctx_s[kSegRows];
    __shared__ KvSharedSeg seg_s[kSegSegs];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, hpg = a.num_heads / a.kv_heads;
    int32_t *ctx = a.num_rows <= kSegRows ? ctx_s : s.own_ctx;  // what each row reads itself (-1: its group is refused)
    KvSharedSeg *seg = s.num_segments <= kSegSegs ? seg_s : s.seg;
    // (parts as in a segment of all rows: near enough for what all own tokens cost)
    const int32_t any_part_min = a.num_rows / a.group * a.kv_heads >= kManyGroups ? kManyPartMin : kPartMin;
    const float own_heads = static_cast<float>(a.kv_heads * ((a.group * hpg + 63) / 64));
    if (threadIdx.x == 0) own_s = 0;
    __syncthreads();
    pdl_wait();
    if (blockIdx.x > 0) {
        if (a.head_dim == 64) split_queries<64>(s, blockIdx.x - 1, gridDim.x - 1);
        else split_queries<128>(s, blockIdx.x - 1, gridDim.x - 1);
        return;
    }
    for (int i = 1 + threadIdx.x; i < 1 + kOwnSms; i += kSegThreads) s.own_sms[i] = 0;
    // every row by itself at first
    float mine = 0.f;
    for (int g = threadIdx.x; g < a.num_rows / a.group; g += kSegThreads) {
        const int row0 = g * a.group;
        int32_t n[kMaxGroup], req[kMaxGroup];
#pragma unroll
        for (int r = 0; r < kMaxGroup; ++r) {
            const int row = row0 + (r < a.group ? r : 0);
            n[r] = s.row_ctx[row];
            req[r] = a.row_req[row];
        }
        bool bad = false;
#pragma unroll
        for (int r = 0; r < kMaxGroup; ++r) bad |= kv_refused(a, n[r], req[r], req[0]);
#pragma unroll
        for (int r = 0; r < kMaxGroup; ++r)
            if (r < a.group) {
                ctx[row0 + r] = bad ? -1 : n[r];
                s.row_begin[row0 + r] = kPartMin;
                s.row_seg[row0 + r] = -1;
            }
        int32_t most = 0;
#pragma unroll
        for (int r = 0; r < kMaxGroup; ++r) most = max(most, n[r]);
        if (!bad) mine += own_cost(s, most, any_part_min);
    }
    mine = warp_sum(mine);
    if (lane == 0) atomicAdd(&own_s, static_cast<unsigned long long>(static_cast<long long>(mine)));
    check_segments(s, tops, [&](int i, int32_t row0, int32_t rows, int32_t shared) {
        KvSharedSeg g = {};
        g.row0 = row0;
        g.rows = rows;
        g.tiles = shared / kTile;
        seg[i] = g;
    });
    __syncthreads();
    // a warp a segment: what all its rows see, and how that is cut
    for (int i = warp; i < s.num_segments; i += kSegThreads / 32) {
        KvSharedSeg g = seg[i];
        const int groups = g.rows / a.group;
        int32_t least = INT32_MAX, lead = INT32_MAX, live = 0;
        for (int j = lane; j < groups; j += 32) {
            bool sees = false;
            for (int r = g.row0 + j * a.group; r < g.row0 + (j + 1) * a.group; ++r) {
                const int32_t n = ctx[r];
                if (n > 0) {
                    least = min(least, n);
                    sees = true;
                }
            }
            live += sees;
            if (sees) lead = min(lead, g.row0 + j * a.group);
        }
        least = __reduce_min_sync(0xffffffffu, least);
        lead = __reduce_min_sync(0xffffffffu, lead);
        live = __reduce_add_sync(0xffffffffu, live);
        g.tiles = live >= 2 ? min(least / kTile, g.tiles) : 0;
        if ((live - 1ll) * g.tiles * kTile * token_bytes(a) < s.least_saved) g.tiles = 0;
        if (g.tiles > 0) {
            const int cols = g.rows * hpg;
            g.blocks = (cols + 2 * kTile - 1) / (2 * kTile);
            g.req = a.row_req[lead];
            const bool narrow = cols - (g.blocks - 1) * 2 * kTile <= kTile;  // the last block is of one chain's columns
            const int each = g.blocks == 1 && narrow ? 1 : 2;                // tiles of one chain that a tile makes
            const int32_t part_min = live * a.kv_heads >= kManyGroups ? kManyPartMin : kPartMin;
            float own = 0.f, before = 0.f;
            for (int j = lane; j < groups; j += 32) {
                int32_t most = 0;
                for (int r = g.row0 + j * a.group; r < g.row0 + (j + 1) * a.group; ++r) {
                    const int32_t n = ctx[r];
                    s.row_begin[r] = g.tiles * kTile + part_min;
                    if (n > 0) {
                        ctx[r] = n - g.tiles * kTile;
                        s.row_seg[r] = i;
                    }
                    most = max(most, n);
                }
                before += own_cost(s, most, any_part_min);
                own += own_cost(s, most - g.tiles * kTile, part_min);
            }
            own = warp_sum(own);
            before = warp_sum(before);
            if (lane == 0) atomicAdd(&own_s, static_cast<unsigned long long>(static_cast<long long>(own - before)));
            // The parts that end first, if the call's other rows are as these and a CTA runs an item at a time (so a row's
            // bits depend on its segment and the call's shapes); the fewest of those that are as good, or, beside other
            // segments, the most of those within an eighth
            const int units = a.kv_heads * g.blocks, most = min(shared_parts_cap(units), max(1, g.tiles / kMinTiles));
            const float alike = __fdiv_rn(static_cast<float>(a.num_rows), static_cast<float>(g.rows));
            const float all = static_cast<float>(units) * alike;
            float sms = kSharedCtas;
            if (s.beside) {
                const float work = all * static_cast<float>(g.tiles * each) + kSharedCtas * kItemTiles;
                sms = rintf(kSharedCtas * __fdiv_rn(work, work + own * own_heads * alike));
                sms = fminf(fmaxf(sms, kFewestSms), kMostSms);
            }
            const float join = static_cast<float>(g.rows) * static_cast<float>(a.num_heads * a.head_dim) * 0x1p-18f;
            const auto time_of = [&](int p) {
                const float item = static_cast<float>((g.tiles + p - 1) / p * each + kItemTiles);
                return rounds_of(all * static_cast<float>(p), sms) * item + join * static_cast<float>(p);
            };
            float best = INFINITY;
            for (int p = 1 + lane; p <= most; p += 32) best = fminf(best, time_of(p));
            best = __uint_as_float(__reduce_min_sync(0xffffffffu, __float_as_uint(best)));
            int first = INT32_MAX, last = 0;
            for (int p = 1 + lane; p <= most; p += 32) {
                const float time = time_of(p);
                if (time <= 1.0001f * best) first = min(first, p);
                if (time <= 1.125f * best) last = p;
            }
            first = __reduce_min_sync(0xffffffffu, first);
            last = __reduce_max_sync(0xffffffffu, last);
            g.parts = max(1, min(s.num_segments > 1 ? last : first, most));
            g.entries = narrow ? 2 * g.parts : g.parts;
            g.cost = (g.tiles + g.parts - 1) / g.parts * each + kItemTiles;
        }
        if (lane == 0) seg[i] = g;
    }
    __syncthreads();
    // (not before: kv_attention*'s CTAs are to find every SM free, for two of them on each)
    pdl_launch_dependents();
    __shared__ int64_t total_s;
    if (warp == 0) {
        // Where there is a CTA for each item, one each, whatever they cost (by cost a CTA may have two that are short, and
        // take longer than for the longest: verify rows of 16 requests over prompts of 8K to 16K 64 us, 62.9)
        int64_t items = 0, work = 0;
        int32_t longest = 0;
        for (int i = lane; i < s.num_segments; i += 32) {
            const int64_t n = static_cast<int64_t>(a.kv_heads) * seg[i].blocks * seg[i].parts;
            items += n;
            work += n * seg[i].cost;
            if (n > 0) longest = max(longest, seg[i].cost);
        }
        items = warp_sum(items);
        work = warp_sum(work);
        longest = __reduce_max_sync(0xffffffffu, longest);
        int sms = kSharedCtas;
        if (s.beside && work > 0) {
            const float own = static_cast<float>(static_cast<long long>(own_s)) * own_heads;
            const float count = static_cast<float>(items), top = static_cast<float>(longest), sum = static_cast<float>(work);
            const bool alike = work == items * longest;
            const auto shared_time = [&](float n) {
                return alike ? rounds_of(count, n) * top : count <= n ? top : __fdividef(sum, n) + top;
            };
            float best = shared_time(kSharedCtas) + own * (1.f / kSharedCtas) + 14.f;  // one after the other
            for (int n = kFewestSms + lane; n <= kMostSms; n += 32) {
                const float time = fmaxf(shared_time(n), __fdividef(own, static_cast<float>(kSharedCtas - n)) + 5.f);
                if (time < best) {
                    best = time;
                    sms = n;
                }
            }
            const float least = __uint_as_float(__reduce_min_sync(0xffffffffu, __float_as_uint(best)));
            sms = __reduce_min_sync(0xffffffffu, best == least ? sms : kSharedCtas);
        }
        if (lane == 0) {
            sms_s = sms;
            s.own_sms[0] = sms < kSharedCtas ? kSharedCtas - sms : kSharedCtas;
        }
        int64_t entry0 = 0, cost0 = 0;
        for (int i0 = 0; i0 < s.num_segments; i0 += 32) {
            const int i = i0 + lane;
            int64_t entries = 0, cost = 0;
            if (i < s.num_segments) {
                KvSharedSeg &g = seg[i];
                if (items <= sms) g.cost = 1;
                entries = static_cast<int64_t>(g.rows) * g.entries;
                cost = static_cast<int64_t>(a.kv_heads) * g.blocks * g.parts * g.cost;
            }
            int64_t e = entries, c = cost;
            for (int o = 1; o < 32; o <<= 1) {
                const int64_t u = __shfl_up_sync(0xffffffffu, e, o), v = __shfl_up_sync(0xffffffffu, c, o);
                if (lane >= o) {
                    e += u;
                    c += v;
                }
            }
            if (i < s.num_segments) {
                seg[i].entry0 = entry0 + e - entries;
                seg[i].cost0 = cost0 + c - cost;
            }
            entry0 += __shfl_sync(0xffffffffu, e, 31);
            cost0 += __shfl_sync(0xffffffffu, c, 31);
        }
        if (lane == 0) total_s = cost0;
    } else if (ctx == ctx_s) {
        for (int r = threadIdx.x - 32; r < a.num_rows; r += kSegThreads - 32) s.own_ctx[r] = ctx_s[r];
    }
    __syncthreads();
    if (seg == seg_s)
        for (int i = threadIdx.x; i < s.num_segments; i += kSegThreads) s.seg[i] = seg_s[i];
    // a CTA takes the items that start within its share of the cost
    if (threadIdx.x < kSharedCtas) {
        const int sms = sms_s;
        const int64_t from = total_s * threadIdx.x / sms;
        KvSharedCta w = {-1, 0, total_s * (threadIdx.x + 1) / sms};
        int lo = 0, hi = s.num_segments;  // the last segment that begins at or before `from`
        while (hi - lo > 1) {
            const int m = (lo + hi) >> 1;
            if (seg[m].cost0 <= from) lo = m;
            else hi = m;
        }
        int64_t at = w.end;
        for (int i = lo; i < s.num_segments; ++i) {
            const KvSharedSeg &g = seg[i];
            const int items = a.kv_heads * g.blocks * g.parts;
            if (items == 0) continue;
            w.item = from > g.cost0 ? static_cast<int>((from - g.cost0 + g.cost - 1) / g.cost) : 0;
            if (w.item >= items) continue;
            w.seg = i;
            at = g.cost0 + static_cast<int64_t>(w.item) * g.cost;
            break;
        }
        if (at >= w.end || static_cast<int>(threadIdx.x) >= sms) w.seg = -1;
        s.cta[threadIdx.x] = w;
    }
}

// ------------------------------------------------------------------ the shared tokens

// A CTA's items: those that start within its share of the cost of all.
struct SharedCursor {
    KvSharedSeg g;
    int s, i, items;        // segment, item of it
    int64_t at, end;        // cost before the item; where this CTA's share ends
    int head, part, block;  // KV head
    int t0, tiles;          // first tile, and how many
    bool wide;              // a chain each for the two halves of the columns

    __device__ __forceinline__ bool place(const KvSharedArgs &a) {
        if (at >= end) return false;
        const int per = g.parts * g.blocks;
        head = i / per;
        const int rest = i - head * per;
        block = rest / g.parts;
        part = rest - block * g.parts;
        // (at most 152 parts of at most 2^23 tiles)
        t0 = static_cast<int>(static_cast<uint32_t>(part * g.tiles) / g.parts);
        tiles = static_cast<int>(static_cast<uint32_t>((part + 1) * g.tiles) / g.parts) - t0;
        wide = g.rows * a.a.hpg - block * 2 * kTile > kTile;
        return true;
    }
    __device__ __forceinline__ void load(const KvSharedArgs &a) {
        g = read_segment(a.seg + s);
        items = a.a.kv_heads * g.blocks * g.parts;
    }
    __device__ __forceinline__ bool first(const KvSharedArgs &a) {
        const int4 w = early_read(reinterpret_cast<const int4 *>(a.cta + blockIdx.x));  // (a KvSharedCta)
        if (w.x < 0) return false;
        s = w.x;
        i = w.y;
        end = static_cast<int64_t>(static_cast<uint32_t>(w.w)) << 32 | static_cast<uint32_t>(w.z);
        load(a);
        at = g.cost0 + static_cast<int64_t>(i) * g.cost;
        return place(a);
    }
    __device__ __forceinline__ bool skip(const KvSharedArgs &a) {  // to the next segment's first item
        i = 0;
        do {
            if (++s >= a.num_segments) return false;
            load(a);
        } while (items == 0);
        at = g.cost0;
        return place(a);
    }
    __device__ __forceinline__ bool next(const KvSharedArgs &a) {
        at += g.cost;
        if (++i >= items) return at < end && skip(a);
        return place(a);
    }
    // steps of a chain: every tile, or every other one
    __device__ __forceinline__ int steps(int chain) const { return wide ? tiles : (tiles + 1 - chain) / 2; }
};

template <bool kFp8, int D>
struct SharedCfg {
    static constexpr int kRowBytes = D * (kFp8 ? 1 : 2);
    static constexpr int kBoxBytes = kRowBytes < 128 ? kRowBytes : 128;
    static constexpr int kBoxes = kRowBytes / kBoxBytes;
    static constexpr int kPlane = kTile * kBoxBytes;                  // one box column of a tile
    static constexpr int kSlotBytes = kTile * kRowBytes;              // K or V of a tile as stored
    static constexpr int kQBytes = kTile * D * 2;                     // a chain's columns, in bf16 or as two e4m3 terms
    static constexpr int kVBytes = kFp8 ? kTile * D * 2 : 0;          // V of a tile in fp16
    static constexpr int kVBufs = kFp8 ? 3 : 0;
    // A ring for K and one for V, each of an even number of slots: a tile's are those of every other tile.
    static constexpr int kRoom = (229376 - 2 * kQBytes - kVBufs * kVBytes) / (2 * kSlotBytes) / 2 * 2;
    static constexpr int kSlots = kRoom > 6 ? 6 : kRoom;
    static_assert(kSlots >= 2, "rings");
    static constexpr int kWarpgroups = kFp8 ? 4 : 3;  // two of softmax, (one that converts V,) the producer and the issuer
    static constexpr int kThreads = 128 * kWarpgroups;
    static constexpr int kRun = 16;                // scores in registers at a time (32: bf16 67.0 us in the place of 65.0)
    static constexpr uint32_t kTmemO = 2 * kTile;  // the chains' scores, then their outputs
    static constexpr int OFF_V = 2 * kQBytes;
    static constexpr int OFF_RING = OFF_V + kVBufs * kVBytes;
    static constexpr int OFF_BARS = OFF_RING + 2 * kSlots * kSlotBytes;
    static constexpr int kNumBars = 4 * kSlots + 1 + 2 * 6 + 2 * 3;
    static constexpr int OFF_MISC = OFF_BARS + kNumBars * 8;
    static constexpr int kSmemBytes = OFF_MISC + 16 + 1024;
    static_assert(kSmemBytes <= 232448, "shared memory");
    // A base leaves the largest weight that it was made for at 2^kBias, so that fp16's steps are 2^-31 of it, and moves
    // when a tile's weights make up more than kMost (fp16 holds 65504; 128 of 2^7 are 2^14).
    static constexpr float kBias = kFp8 ? 7.0f : 0.0f, kMost = kFp8 ? 32768.0f : 1048576.0f;
};

// 16 bytes to shared memory while the thread goes on; zeros unless `there`.
__device__ __forceinline__ void copy16(void *dst, const void *src, bool there) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(there ? 16 : 0)
                 : "memory");
}

// A warp's 32 columns (lane l: column l's 2 D bytes at `src`, NULL behind the last) into the chain's image, from row
// `n0` on: bf16, 64 dims to a 128-byte row, or e4m3 terms, hi and then lo.  D / 8 lanes take a column, so that the warp
// reads whole runs of memory (a thread a column: 11,000 cycles), all of it on its way at once; in a rolled loop, for code
// that runs once waits for its way in.
template <bool kFp8, int D>
__device__ __forceinline__ void put_queries(uint8_t *img, const uint8_t *src, int n0, int lane) {
    constexpr int kLanes = D / 8, kCols = 32 / kLanes;  // of a column; of a turn
    const int unit = lane % kLanes, sub = lane / kLanes;
#pragma unroll 1
    for (int n = sub; n < 32; n += kCols) {
        const auto *q = reinterpret_cast<const uint8_t *>(
            __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(src), n));
        const int r = n0 + n;
        const uint32_t at = kFp8 && D == 64 ? (unit >> 2) * (kTile * 64) + r * 64 + (((unit & 3) ^ (r >> 1 & 3)) << 4)
                                            : (unit >> 3) * (kTile * 128) + fp8mla::sw128(r, unit & 7);
        copy16(img + at, q != nullptr ? q + unit * 16 : img, q != nullptr);
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
}

// Four e4m3 codes as two fp16 pairs (exact).
__device__ __forceinline__ void codes_to_f16(uint32_t v, uint32_t &lo, uint32_t &hi) {
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(v));
}

template <bool kFp8, int D>
__global__ void __launch_bounds__(SharedCfg<kFp8, D>::kThreads, 1)
    kv_shared_kernel(const __grid_constant__ CUtensorMap kv_map, const __grid_constant__ KvSharedArgs s) {
    using C = SharedCfg<kFp8, D>;
    constexpr int NS = C::kSlots;
    const KvAttnArgs &a = s.a;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + C::OFF_BARS);  // [2 NS] K, then V landed
    uint64_t *empty = full + 2 * NS;                                    // [2 NS] it has been used
    uint64_t *q_full = empty + 2 * NS;                                      // [2] a chain's queries are in place
    uint64_t *q_empty = q_full + 2;                                     // the item's scores are done
    uint64_t *s_full = q_empty + 1;                                     // [2] a chain's scores in TMEM
    uint64_t *p_full = s_full + 2;                                      // [2] its weights in their place
    uint64_t *o_full = p_full + 2;                                      // [2] its item's output is done
    uint64_t *v_full = o_full + 2;                                      // [3] V in fp16
    uint64_t *v_empty = v_full + 3;                                     // [3] and its product done
    uint64_t *my_turn = v_empty + 3;                                    // [2] the other chain's warp has issued
    uint64_t *drained = my_turn + 2;                                    // [2] after a wait gave up: no MMA is left
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + C::OFF_MISC);
    volatile int *abort = reinterpret_cast<volatile int *>(smem + C::OFF_MISC + 4);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, wg = warp >> 2;
    constexpr int kProducer = 4 * (C::kWarpgroups - 1), kIssuer = kProducer + 2;  // two warps each
    if (threadIdx.x == 0) {
        *abort = 0;
        for (int i = 0; i < 2 * NS; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], kFp8 && i >= NS ? 4 : 2);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&q_full[i], 4);
            mbar_init(&s_full[i], 1);
            mbar_init(&p_full[i], 4);
            mbar_init(&o_full[i], 1);
            mbar_init(&my_turn[i], 1);
            mbar_init(&drained[i], 1);
        }
        for (int i = 0; i < 3; ++i) {
            mbar_init(&v_full[i], 4);
            mbar_init(&v_empty[i], 2);
        }
        mbar_init(q_empty, 2);
        fence_mbar_init();
        prefetch_tensormap(&kv_map);
    }
    if (warp == kIssuer) {
        tmem_alloc(tmem_slot, 512);
        tmem_relinquish();
        tc_fence_before();
    }
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    // What this kernel reads was complete when the one before it (kv_attention*.cu), which writes nothing that this one
    // reads or writes, passed its own wait and let this one start.  So it begins while that one ends, and waits for it at
    // the end, for the join's sake.
    pdl_launch_dependents();
    SharedCursor w;
    bool more = w.first(s);
    if (wg >= 2) {
        if (kFp8 && wg == 2) {
            // ---- V's codes as fp16: thread = token
            const int t = threadIdx.x & 127;
            uint32_t n = 0;  // tiles
            bool ok = true;
            for (; more && ok; more = w.next(s)) {
                for (int i = 0; i < w.tiles && ok; ++i, ++n) {
                    const uint32_t slot = NS + n % NS, buf = n % 3;
                    ok = wait_mbar_warp(&full[slot], n / NS & 1, abort) &&
                         wait_mbar_warp(&v_empty[buf], (n / 3 & 1) ^ 1, abort);
                    if (!ok) break;
                    const uint8_t *from = smem + C::OFF_RING + slot * C::kSlotBytes;
                    uint8_t *to = smem + C::OFF_V + buf * C::kVBytes;
#pragma unroll
                    for (int u = 0; u < D / 16; ++u) {
                        const uint4 v = *reinterpret_cast<const uint4 *>(
                            from + (D == 128 ? fp8mla::sw128(t, u) : static_cast<uint32_t>(t * 64 + ((u ^ (t >> 1 & 3)) << 4))));
                        uint4 x, y;
                        codes_to_f16(v.x, x.x, x.y);
                        codes_to_f16(v.y, x.z, x.w);
                        codes_to_f16(v.z, y.x, y.y);
                        codes_to_f16(v.w, y.z, y.w);
                        uint8_t *plane = to + (u >> 2) * (kTile * 128);
                        *reinterpret_cast<uint4 *>(plane + fp8mla::sw128(t, 2 * u & 7)) = x;
                        *reinterpret_cast<uint4 *>(plane + fp8mla::sw128(t, (2 * u & 7) + 1)) = y;
                    }
                    fence_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(&v_full[buf]);
                        mbar_arrive(&empty[slot]);
                    }
                }
            }
            if (!ok) gave_up(abort, a.status);
        } else if (warp < kIssuer) {
            // ---- K, and V by another warp (in one order V, whose place is taken until its weights are done, would hold up
            // the next K): a tile is `boxes` runs of tokens by kBoxes columns, one a lane
            const int v = __shfl_sync(0xffffffffu, warp - kProducer, 0);
            const int box_rows = a.page_size, boxes = kTile >> a.page_shift;
            const int b = lane / C::kBoxes, x = lane % C::kBoxes;
            uint32_t turn = 0;  // tiles
            bool go = true;
            for (; more && go; more = w.next(s)) {
                const int32_t *table = a.block_table + static_cast<int64_t>(w.g.req) * a.bt_stride;
                const int page0 = w.t0 << 7 >> a.page_shift, pages = w.tiles << 7 >> a.page_shift;
                auto load_ids = [&](int p) { return p + lane < pages ? early_read(table + page0 + p + lane) : 0; };
                int batch = 0;  // page ids batch .. batch + 31 of the item are in `ids`, one per lane
                int32_t ids = load_ids(0), ids_next = load_ids(32);
                for (int i = 0; i < w.tiles; ++i, ++turn) {
                    const int p = i << 7 >> a.page_shift;
                    if (p >= batch + 32) {
                        batch += 32;
                        ids = ids_next;
                        ids_next = load_ids(batch + 32);
                    }
                    int32_t id = __shfl_sync(0xffffffffu, ids, (p + min(b, boxes - 1) - batch) & 31);
                    if (b < boxes && (id < 0 || id >= a.num_pages)) {
                        report(a.status, DSA_ERR_BOUNDS);
                        id = 0;
                    }
                    const int y = ((id * a.kv_heads + w.head) * 2 + v) * a.page_size;
                    const uint32_t slot = v * NS + turn % NS;
                    if (!wait_mbar_warp(&empty[slot], (turn / NS & 1) ^ 1, abort)) {
                        gave_up(abort, a.status);
                        go = false;
                        break;
                    }
                    if (lane == 0) mbar_arrive_expect_tx(&full[slot], C::kSlotBytes);
                    __syncwarp();
                    if (b < boxes)
                        tma_load_2d(smem + C::OFF_RING + slot * C::kSlotBytes + x * C::kPlane + b * box_rows * C::kBoxBytes,
                                    &kv_map, &full[slot], x * C::kBoxBytes, y);
                }
            }
            if (*abort && lane == 0) {  // leave no copy in flight behind
                for (uint32_t i = turn > NS ? turn - NS : 0; i < turn; ++i) {
                    const long long t0 = clock64();
                    while (!mbar_try_wait(&full[v * NS + i % NS], i / NS & 1) && clock64() - t0 < kWaitTimeoutCycles) {
                    }
                }
            }
        } else {
            // ---- the products, a warp a chain: an MMA's issue lasts as long as its passage, and what lies between two runs
            // of MMAs (1,000 cycles of commits and waits) is the other warp's time.  The warps take turns, so that one
            // chain's products stay beside the other's softmax: left to themselves the chains fall into step (3,690
            // cycles for a tile of both, in turns 2,450; one warp for both 3,150).  MMAs of a thread run in the order of
            // their issue, so a chain's next scores, which take the place of its weights, are right behind the product that
            // reads those.  A warp goes through all of this together, so that descriptors stay in uniform registers, and
            // one lane issues.
            // (Of tiles that the chains share out a warp waits for its own alone.  The slots of every other tile are the
            // same ones, V's conversions come in order, and all of an item's tiles have landed when the next begins: so the
            // phase before an awaited one is over, and a barrier's parity tells.)
            constexpr uint32_t kIdescS = make_idesc(kTile, kTile, kFp8 ? 0 : 1, kFp8 ? 0 : 1, false, false);
            constexpr uint32_t kIdescO = make_idesc(kTile, D, kFp8 ? 0 : 1, kFp8 ? 0 : 1, false, true);
            const uint32_t base = __shfl_sync(0xffffffffu, smem_u32(smem), 0), ring = base + C::OFF_RING;
            const uint32_t t_mem = __shfl_sync(0xffffffffu, tmem, 0);
            const int c = __shfl_sync(0xffffffffu, warp - kIssuer, 0);
            const uint32_t st = t_mem + c * kTile, ot = t_mem + C::kTmemO + c * D;
            const bool lead = elect_one();
            uint32_t n = 0, items = 0, p_count = 0, turns = 0;  // tiles before the item, items, products, turns taken
            bool ok = true;
            for (; more && ok; more = w.next(s), ++items) {
                const bool wide = __shfl_sync(0xffffffffu, w.wide, 0);
                const int tiles = __shfl_sync(0xffffffffu, w.tiles, 0);
                const int most = wide ? tiles : (tiles + 1) / 2, steps = wide ? tiles : (tiles + 1 - c) / 2;
                auto tile_of = [&](int j) { return n + static_cast<uint32_t>(wide ? j : 2 * j + c); };
                const uint32_t q = base + (wide ? c : 0) * C::kQBytes;
                const uint64_t qd = !kFp8 || D == 128 ? sdesc_sw128(q, 16, 1024) : sdesc_sw64(q);
                auto used = [&](uint64_t *bar) {  // two arrivals: one of each chain, or both of the only one
                    if (!wide) mbar_arrive(bar);
                    mma_commit(bar);
                };
                ok = wait_mbar_warp(&q_full[0], items & 1, abort) && wait_mbar_warp(&q_full[1], items & 1, abort);
                // the product of step j (from 0 on) and the scores of step j + 1 (where there is one)
                for (int j = -1; j < most && ok; ++j) {
                    const uint32_t tile = tile_of(j), v_slot = NS + tile % NS, buf = tile % 3;
                    const uint32_t k_tile = tile_of(j + 1), k_slot = k_tile % NS;
                    const bool product = j >= 0 && j < steps, next = j + 1 < steps;
                    const uint32_t k = ring + k_slot * C::kSlotBytes;
                    const uint32_t v = kFp8 ? base + C::OFF_V + buf * C::kVBytes : ring + v_slot * C::kSlotBytes;
                    const uint64_t vd = sdesc_sw128(v, kTile * 128, 1024);
                    const uint64_t kd = !kFp8 || D == 128 ? sdesc_sw128(k, 16, 1024) : sdesc_sw64(k);
                    if (next) ok = ok && wait_mbar_warp(&full[k_slot], k_tile / NS & 1, abort);
                    if (product)
                        ok = ok && (kFp8 ? wait_mbar_warp(&v_full[buf], tile / 3 & 1, abort)
                                         : wait_mbar_warp(&full[v_slot], tile / NS & 1, abort));
                    ok = ok && wait_mbar_warp(&my_turn[c], (turns++ & 1) ^ (c == 0 ? 1 : 0), abort);
                    if (product) ok = ok && wait_mbar_warp(&p_full[c], p_count++ & 1, abort);
                    if (!ok) break;
                    tc_fence_after();
                    if (lead) {
                        if (product) {
                            const uint32_t add = j > 0;
#pragma unroll
                            for (int i = 0; i < kTile / 16; ++i)
                                mma_f16_ts(ot, st + i * 8, vd + i * 128, kIdescO, i > 0 ? 1u : add);
                        }
                        if (next) {
                            if constexpr (kFp8) {
#pragma unroll
                                for (int term = 0; term < 2; ++term)
#pragma unroll
                                    for (int i = 0; i < D / 32; ++i)
                                        mma_f8(st, qd + term * (kTile * D / 16) + i * 2, kd + i * 2, kIdescS, term + i > 0);
                            } else {
#pragma unroll
                                for (int i = 0; i < D / 16; ++i) {
                                    const uint32_t off = (i >> 2) * (kTile * 128 / 16) + (i & 3) * 2;
                                    mma_f16(st, qd + off, kd + off, kIdescS, i > 0);
                                }
                            }
                        }
                        mbar_arrive(&my_turn[1 - c]);
                        if (next) {
                            mma_commit(&s_full[c]);
                            used(&empty[k_slot]);
                        } else if (product) {
                            mma_commit(&o_full[c]);
                        }
                        if (product) used(kFp8 ? &v_empty[buf] : &empty[v_slot]);
                    }
                    __syncwarp();
                }
                if (!ok) break;
                if (lead) mma_commit(q_empty);
                __syncwarp();
                n += static_cast<uint32_t>(tiles);
            }
            if (!ok) gave_up(abort, a.status);
            if (*abort) {  // leave no MMA in flight behind
                if (lead) mma_commit(&drained[c]);
                __syncwarp();
                const long long t0 = clock64();
                while (!mbar_try_wait(&drained[c], 0) && clock64() - t0 < kWaitTimeoutCycles) {
                }
            }
        }
        __syncwarp();
    } else {
        // ---- softmax of chain wg: thread = column
        const int self = threadIdx.x & 127, c = wg;
        const uint32_t quad = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
        const uint32_t st = quad + c * kTile, ot = quad + C::kTmemO + c * D;
        uint32_t s_count = 0, items = 0, outs = 0;
        bool ok = true;
        for (; more && ok; more = w.next(s), ++items) {
            const int hpg = a.hpg, col = w.block * 2 * kTile + (w.wide ? c * kTile : 0) + self;
            const bool real = col < w.g.rows * hpg;
            ok = wait_mbar_warp(q_empty, (items & 1) ^ 1, abort);
            if (!ok) break;
            const int of = w.wide ? c : 0;  // (one image serves two chains of the same columns)
            // this column's row of the segment and head; where its output goes, in outputs of D
            const int row = static_cast<int>(static_cast<uint32_t>(col) / static_cast<uint32_t>(hpg));
            const int head = w.head * hpg + col - row * hpg;
            const int64_t place = (w.g.entry0 + static_cast<int64_t>(row) * w.g.entries + (w.wide ? w.part : 2 * w.part + c)) *
                                      a.num_heads + head;
            const int64_t at = (w.g.row0 + row) * static_cast<int64_t>(a.num_heads) + head;
            const int steps = w.steps(c);
            float scale = a.s_scale;
            if (kFp8 && real) scale *= early_read(s.q_factor + at);
            if (of == c) {
                const uint8_t *src = kFp8 ? s.q_terms + at * (2 * D)
                                          : reinterpret_cast<const uint8_t *>(a.q + (w.g.row0 + row) * a.q_stride +
                                                                              static_cast<int64_t>(head) * D);
                put_queries<kFp8, D>(smem + c * C::kQBytes, real ? src : nullptr, (warp & 3) * 32, lane);
                fence_async_smem();
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&q_full[c]);
            // a score of -inf times the scale: neither zero nor infinity.  Over codes no number in q makes no score
            if (scale == scale) scale = fminf(fmaxf(scale, 1.17549435e-38f), 3.40282347e38f);
            float base = -INFINITY;
            float2 sum = make_float2(0.f, 0.f);
            for (int j = 0; j < steps; ++j, ++s_count) {
                ok = wait_mbar_warp(&s_full[c], s_count & 1, abort);
                if (!ok) break;
                tc_fence_after();
                // P = 2^(scale S - b), kRun tokens at a time with the next ones on their way, into registers: S is
                // overwritten when no weight is too large for b.  A tile's sum tells that as well as its largest would,
                // without one more pass; the largest is looked for where it is, and where there is no base yet.  (Half a
                // tile at a time, with the first half's product beside the second's exponentials: 2,900 cycles for a
                // tile of both chains against 2,820, since the chains' exponentials then meet.)
                uint32_t p[kTile / 2];
                bool moves = base == -INFINITY, moved = false;
#pragma unroll 1
                while (true) {  // (three times at most: a column's base moves once a tile)
                    if (__any_sync(0xffffffffu, moves)) {
                        float top = -INFINITY;
#pragma unroll 1
                        for (int i = 0; i < kTile; i += 32) {
                            uint32_t h[32];
                            tmem_ld32(st + i, h);
                            tmem_ld_wait();
                            reg_fence(h);
#pragma unroll
                            for (int k = 0; k < 32; ++k) top = fmaxf(top, __uint_as_float(h[k]));
                        }
                        top = top * scale - C::kBias;  // (a positive factor)
                        moved |= moves;
                        moves = moves && top > base;
                        const float f = moves ? ex2(base - top) : 1.f;
                        if (moves) base = top;
                        sum.x *= f;
                        sum.y *= f;
                        // (this tile's scores are done, so the products before them are: O is at rest)
                        if (j > 0 && __any_sync(0xffffffffu, moves)) {
#pragma unroll 1
                            for (int i = 0; i < D; i += 16) {
                                uint32_t o[16];
                                tmem_ld16(ot + i, o);
                                tmem_ld_wait();
                                reg_fence(o);
#pragma unroll
                                for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
                                tmem_st16(ot + i, o);
                            }
                        }
                    }
                    const float nb = base == -INFINITY ? 0.f : -base;
                    const float2 sc2 = make_float2(scale, scale), nb2 = make_float2(nb, nb);
                    float2 t0 = make_float2(0.f, 0.f), t1 = make_float2(0.f, 0.f);
                    constexpr int kRun = C::kRun;
                    static_assert(kRun == 16, "load");
                    uint32_t h[2][kRun];
                    auto load = [&](int i) { tmem_ld16(st + kRun * i, h[i & 1]); };
                    load(0);
#pragma unroll
                    for (int i = 0; i < kTile / kRun; ++i) {
                        tmem_ld_wait();
                        reg_fence(h[i & 1]);
                        if (i + 1 < kTile / kRun) load(i + 1);
#pragma unroll
                        for (int k = 0; k < kRun; k += 2) {
                            float2 x = __ffma2_rn(
                                make_float2(__uint_as_float(h[i & 1][k]), __uint_as_float(h[i & 1][k + 1])), sc2, nb2);
                            x.x = ex2(x.x);
                            x.y = ex2(x.y);
                            if (k & 2) t1 = __fadd2_rn(t1, x);
                            else t0 = __fadd2_rn(t0, x);
                            p[(kRun * i + k) / 2] = kFp8 ? pack_f16(x.x, x.y) : pack_bf16(x.x, x.y);
                        }
                    }
                    t0 = __fadd2_rn(t0, t1);
                    moves = !moved && t0.x + t0.y > C::kMost;
                    if (!__any_sync(0xffffffffu, moves)) {
                        sum = __fadd2_rn(sum, t0);
                        break;
                    }
                }
                tmem_st32(st, *reinterpret_cast<uint32_t(*)[32]>(p));
                tmem_st32(st + 32, *reinterpret_cast<uint32_t(*)[32]>(p + 32));
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&p_full[c]);
            }
            if (!ok) break;
            // ---- the item's output, by way of the chain's queries' place: a warp writes whole runs of memory (a thread a
            // column: 5,400 cycles)
            const float total = sum.x + sum.y;
            if (real) s.sml[place] = make_float2(part_base(base, total), total);
            if (steps > 0) {
                ok = wait_mbar_warp(&o_full[c], outs & 1, abort);
                ++outs;
            }
            // (the other chain's scores read the image too)
            if (of == c && !w.wide) ok = ok && wait_mbar_warp(q_empty, items & 1, abort);
            if (!ok) break;
            tc_fence_after();
            // kDims dims of the warp's 32 columns at a time, where its own part of the image is: another warp of the chain
            // may be at the next item's queries already (a barrier between them would wait for a warp that gave up)
            constexpr int kDims = D / 2, kUnits = kDims / 4, kCols = 32 / kUnits;  // 16-byte units of a column, columns a turn
            constexpr int kPlanes = kFp8 || D == 128 ? 2 : 1, kRows = 32 / kPlanes;  // of the image
            uint8_t *stage = smem + c * C::kQBytes + (warp & 3) * (C::kQBytes / 4 / kPlanes);
            const auto stage_at = [&](int n, int unit) {
                return reinterpret_cast<uint4 *>(stage + n / kRows * (C::kQBytes / kPlanes) + n % kRows * (kDims * 4) +
                                                 ((unit ^ (n & 7)) << 4));
            };
#pragma unroll 1
            for (int d0 = 0; d0 < D; d0 += kDims) {
                __syncwarp();
#pragma unroll 1
                for (int i = 0; i < kDims; i += 16) {
                    uint32_t o[16];
                    if (steps > 0) {
                        tmem_ld16(ot + d0 + i, o);
                        tmem_ld_wait();
                        reg_fence(o);
                    } else {  // (no tile for the second chain)
#pragma unroll
                        for (int k = 0; k < 16; ++k) o[k] = 0u;
                    }
#pragma unroll
                    for (int k = 0; k < 16; k += 4)
                        *stage_at(lane, (i + k) / 4) = make_uint4(o[k], o[k + 1], o[k + 2], o[k + 3]);
                }
                __syncwarp();
                const int u = lane % kUnits;
#pragma unroll 4
                for (int n0 = 0; n0 < 32; n0 += kCols) {
                    const int n = n0 + lane / kUnits;
                    const int64_t at = __shfl_sync(0xffffffffu, real ? place : -1, n);
                    if (at >= 0) *reinterpret_cast<uint4 *>(s.so + at * D + d0 + 4 * u) = *stage_at(n, u);
                }
            }
            __syncwarp();
            tc_fence_before();
        }
        if (!ok) gave_up(abort, a.status);
    }
    __syncthreads();
    if (warp == kIssuer) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
    pdl_wait();
}

// ------------------------------------------------------------------ the parts of a (row, head)

// A row's own parts, then the shared ones.  kWarps warps take a (row, head): one, where there are enough of those, else
// four, which share out the parts.  D / 4 lanes take a part, four dims each.
//   us of a call over 32K tokens, 32 heads of 128    one warp, four
//     bf16   4 rows   128 (row, head)                37.0  28.3
//           16        512                            34.1  31.8
//           31        992                            37.0  34.5
//           40      1,280                            45.7  45.7
//           64      2,048                            45.2  50.3
//     FP8   31        992                            41.8  38.8
//           64      2,048                            47.3  52.3
constexpr int kJoinThreads = 128;
constexpr int64_t kJoinPairs = 1024;

template <int D, int kWarps>
__global__ void __launch_bounds__(kJoinThreads) kv_join_kernel(const __grid_constant__ KvSharedArgs s) {
    constexpr int kLanes = D / 4, kAt = 32 / kLanes;  // lanes of a part, parts a turn of a warp
    constexpr int kPairs = kJoinThreads / 32 / kWarps;
    __shared__ float4 x_s[kWarps > 1 ? kJoinThreads : 1];
    __shared__ float2 t_s[kWarps > 1 ? kWarps : 1];
    const KvAttnArgs &a = s.a;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, mine = warp % kWarps;
    // (early_reads of what kv_segments_kernel wrote, and of the call's rows)
    const int64_t at = static_cast<int64_t>(blockIdx.x) * kPairs + warp / kWarps;
    if (kWarps == 1 && at >= static_cast<int64_t>(a.num_rows) * a.num_heads) return;
    const int row = static_cast<int>(at / a.num_heads), head = static_cast<int>(at - static_cast<int64_t>(row) * a.num_heads);
    int req;
    bool bad;
    const int my_ctx = kv_load_group<true>(a, row / a.group * a.group, lane, req, bad);
    const int ctx = __reduce_max_sync(0xffffffffu, my_ctx);
    const int own = ctx > 0 ? kv_parts(ctx, kv_part_shift(ctx, a.parts_shift, kv_part_min(early_read(a.row_begin + row)))) : 0;
    int parts = own;
    int64_t entry = 0;  // the first shared part
    const int32_t seg = early_read(s.row_seg + row);
    if (seg >= 0) {
        const KvSharedSeg g = read_segment(s.seg + seg);
        const int r = row - g.row0, block = (r * a.hpg + head % a.hpg) / (2 * kTile);
        const bool wide = g.rows * a.hpg - block * 2 * kTile > kTile;
        parts += wide ? g.parts : 2 * g.parts;
        entry = g.entry0 + static_cast<int64_t>(r) * g.entries;
    }
    pdl_wait();
    pdl_launch_dependents();
    const int d = lane % kLanes, sub = lane / kLanes;
    const float4 *po = reinterpret_cast<const float4 *>(a.part_o + at * a.parts_bound * D) + d;
    const float4 *so = reinterpret_cast<const float4 *>(s.so + (entry * a.num_heads + head) * D) + d;
    const int64_t so_step = static_cast<int64_t>(a.num_heads) * kLanes;
    const auto ml_at = [&](int p) {
        return p >= parts ? make_float2(-INFINITY, 0.f)
                          : p < own ? a.part_ml[at * a.parts_bound + p] : s.sml[(entry + p - own) * a.num_heads + head];
    };
    // 32 parts at a time, this warp's first: lane l holds the base and sum of part p0 + l
    float b = -INFINITY, total = 0.f;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int p0 = 32 * mine; p0 < parts; p0 += 32 * kWarps) {
        const float2 ml = ml_at(p0 + lane);
        float top = ml.x;
#pragma unroll
        for (int i = 16; i > 0; i >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, i));
        top = fmaxf(top, b);
        const float b0 = top == -INFINITY ? 0.f : top, back = ex2(b - b0);
        b = top;
        const float f = ex2(ml.x - b0);
        total = total * back + ml.y * f;  // (of this lane's parts; added up below)
        x.x *= back;
        x.y *= back;
        x.z *= back;
        x.w *= back;
        const int n = min(32, parts - p0);
#pragma unroll 1
        for (int i = 0; i < n; i += 8 * kAt) {
            float4 y[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const int p = p0 + i + k * kAt + sub;
                y[k] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (p < p0 + n) y[k] = p < own ? po[static_cast<int64_t>(p) * kLanes] : so[(p - own) * so_step];
            }
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const float w = __shfl_sync(0xffffffffu, f, (i + k * kAt + sub) & 31);
                if (i + k * kAt + sub >= n) continue;
                x.x = fmaf(y[k].x, w, x.x);
                x.y = fmaf(y[k].y, w, x.y);
                x.z = fmaf(y[k].z, w, x.z);
                x.w = fmaf(y[k].w, w, x.w);
            }
        }
    }
#pragma unroll
    for (int i = 16; i > 0; i >>= 1) total += __shfl_xor_sync(0xffffffffu, total, i);
#pragma unroll
    for (int i = kLanes; i < 32; i <<= 1) {
        x.x += __shfl_xor_sync(0xffffffffu, x.x, i);
        x.y += __shfl_xor_sync(0xffffffffu, x.y, i);
        x.z += __shfl_xor_sync(0xffffffffu, x.z, i);
        x.w += __shfl_xor_sync(0xffffffffu, x.w, i);
    }
    if constexpr (kWarps > 1) {
        x_s[threadIdx.x] = x;
        if (lane == 0) t_s[warp] = make_float2(b, total);
        __syncthreads();
        if (warp > 0) return;
        float top = b;
#pragma unroll
        for (int i = 1; i < kWarps; ++i) top = fmaxf(top, t_s[i].x);
        const float b0 = top == -INFINITY ? 0.f : top;
        total = 0.f;
        x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int i = 0; i < kWarps; ++i) {
            const float f = ex2(t_s[i].x - b0);
            const float4 v = x_s[32 * i + lane];
            total += t_s[i].y * f;
            x.x += v.x * f;
            x.y += v.y * f;
            x.z += v.z * f;
            x.w += v.w * f;
        }
        b = top;
    }
    const float b0 = b == -INFINITY ? 0.f : b;
    const bool none = total == 0.f;
    const float inv = none ? 0.f : a.v_scale / total;
    if (sub == 0)
        *reinterpret_cast<uint2 *>(a.out + at * D + 4 * d) =
            none ? make_uint2(0u, 0u) : make_uint2(pack_bf16(x.x * inv, x.y * inv), pack_bf16(x.z * inv, x.w * inv));
    if (lane == 0 && a.lse != nullptr) a.lse[at] = none ? -INFINITY : (b0 + log2f(total)) * 0.6931471805599453f;
}

// Checks of kv_segments_kernel alone.
__global__ void __launch_bounds__(kSegThreads, 1) kv_segments_check_kernel(const __grid_constant__ KvSharedArgs s) {
    pdl_wait();
    pdl_launch_dependents();
    __shared__ int32_t tops[kSegThreads / 32];
    check_segments(s, tops, [](int, int32_t, int32_t, int32_t) {});
}

template <int D>
cudaError_t launch_join(const KvSharedArgs &s, cudaStream_t stream) {
    const int64_t pairs = static_cast<int64_t>(s.a.num_rows) * s.a.num_heads;
    if (pairs > 0x7fffffff) return cudaErrorInvalidConfiguration;
    constexpr int kPairs = kJoinThreads / 32;
    if (pairs < kJoinPairs)
        return launch_pdl(kv_join_kernel<D, 4>, dim3(static_cast<unsigned>(pairs)), dim3(kJoinThreads), 0, stream, s);
    return launch_pdl(kv_join_kernel<D, 1>, dim3(static_cast<unsigned>((pairs + kPairs - 1) / kPairs)), dim3(kJoinThreads), 0,
                      stream, s);
}

// ------------------------------------------------------------------ launches

// What a tile of rows' own tokens costs an SM, in tiles of a chain (0.63 us), for one KV head and so many columns.  Measured
// over 16 x 32K tokens, us an SM and tile for 4 / 8 / 16 / 32 / 64 columns: bf16 0.68 / 0.70 / 0.89 / 1.54 / 2.69, of
// head_dim 64 0.41 / 0.41 / 0.50 / 0.84 / 1.51; FP8 0.63 / 0.64 / 0.66 / 0.99 / 1.68, 0.38 / 0.39 / 0.44 / 0.74 / 1.30.
float own_tile(bool fp8, int32_t head_dim, float cols) {
    const float least = head_dim == 128 ? (fp8 ? 1.02f : 1.1f) : fp8 ? 0.62f : 0.66f;
    const float some = head_dim == 128 ? (fp8 ? 0.47f + cols * 0.034f : 0.56f + cols * 0.058f)
                                       : fp8 ? 0.23f + cols * 0.029f : 0.28f + cols * 0.033f;
    return some > least ? some : least;
}

template <bool kFp8, int D>
cudaError_t launch_shared(const KvSharedArgs &s, cudaStream_t stream) {
    using C = SharedCfg<kFp8, D>;
    auto kern = kv_shared_kernel<kFp8, D>;
    static std::atomic<uint64_t> configured{0};
    cudaError_t e = raise_smem_limit(kern, C::kSmemBytes, configured);
    if (e != cudaSuccess) return e;
    CUtensorMap map;
    if (!encode_kv_rows_map(&map, s.a.pool, s.a.pool_rows, C::kRowBytes, s.a.page_size)) return cudaErrorInvalidValue;
    return launch_pdl(kern, dim3(kSharedCtas), dim3(C::kThreads), C::kSmemBytes, stream, map, s);
}

// Shared parts of all (row, head) at most, divided by the heads.  A part has at least rows x heads / 256 items, so
// shared_parts_cap leaves a segment 2 x 4 outputs a row, or 2 x 8 x 152 x 256 / heads in all.
size_t shared_entries(int64_t num_rows, int32_t num_heads, int32_t kv_heads, int32_t max_ctx, int32_t num_segments) {
    const int64_t tiles = max_ctx / kTile, most = tiles / kMinTiles > 1 ? tiles / kMinTiles : 1;
    const int64_t cap = shared_parts_cap(kv_heads) < most ? shared_parts_cap(kv_heads) : most;
    const int64_t by_row = num_rows * 2 * cap;
    const int64_t by_segment = 8 * num_rows + num_segments * (16ll * kSharedCtas * 2 * kTile / num_heads + 1);
    return static_cast<size_t>(by_row < by_segment ? by_row : by_segment);
}

}  // namespace

size_t kv_attention_shared_workspace_bytes(int64_t num_rows, int32_t num_heads, int32_t kv_heads, int32_t head_dim,
                                           int32_t max_ctx, int32_t num_segments, bool fp8) {
    const size_t pairs = fp8 ? static_cast<size_t>(num_rows) * static_cast<size_t>(num_heads) : 0;
    const size_t entries =
        shared_entries(num_rows, num_heads, kv_heads, max_ctx, num_segments) * static_cast<size_t>(num_heads);
    return kv_attention_workspace_bytes(num_rows, num_heads, kv_heads, head_dim, max_ctx, true) +
           3 * align256(static_cast<size_t>(num_rows) * 4) +
           align256(static_cast<size_t>(num_segments) * sizeof(KvSharedSeg)) +
           align256(kSharedCtas * sizeof(KvSharedCta)) + align256((1 + kOwnSms) * 4) +
           align256(entries * static_cast<size_t>(head_dim) * 4) + align256(entries * 8) +
           align256(pairs * 2 * static_cast<size_t>(head_dim)) + align256(pairs * 4);
}

cudaError_t launch_kv_attention_shared(const KvSegmentArgs &seg, KvAttnArgs &a, void *workspace, cudaStream_t stream) {
    if (a.num_rows == 0) return cudaSuccess;
    KvSharedArgs s = {};
    s.first_row = seg.first_row;
    s.shared_ctx = seg.shared_ctx;
    s.num_segments = seg.num_segments;
    const int64_t least = seg.least_saved > 0 ? seg.least_saved : shared_least_bytes(a);
    s.least_saved = seg.least_saved > 0 ? seg.least_saved : least / 2 / seg.num_segments;
    s.row_ctx = a.row_ctx;
    const size_t rows = align256(static_cast<size_t>(a.num_rows) * 4);
    uint8_t *at = static_cast<uint8_t *>(workspace) +
                  kv_attention_workspace_bytes(a.num_rows, a.num_heads, a.kv_heads, a.head_dim, a.max_ctx, true);
    const auto take = [&](size_t bytes) {
        uint8_t *p = at;
        at += bytes;
        return p;
    };
    s.own_ctx = reinterpret_cast<int32_t *>(take(rows));
    s.row_begin = reinterpret_cast<int32_t *>(take(rows));
    s.row_seg = reinterpret_cast<int32_t *>(take(rows));
    s.seg = reinterpret_cast<KvSharedSeg *>(take(align256(static_cast<size_t>(seg.num_segments) * sizeof(KvSharedSeg))));
    s.cta = reinterpret_cast<KvSharedCta *>(take(align256(kSharedCtas * sizeof(KvSharedCta))));
    s.own_sms = reinterpret_cast<int32_t *>(take(align256((1 + kOwnSms) * 4)));
    const int64_t cols = static_cast<int64_t>(a.group) * (a.num_heads / a.kv_heads);
    s.beside = static_cast<int64_t>(a.num_rows / a.group) * a.kv_heads * ((cols + 63) / 64) *
                   kv_parts_bound(a.max_ctx, kv_parts_shift(a.kv_heads)) >
               2 * kSharedCtas;
    s.own_tile = own_tile(a.fp8, a.head_dim, static_cast<float>(cols < 64 ? cols : 64));
    s.own_item = 3.1f;
    const size_t entries = shared_entries(a.num_rows, a.num_heads, a.kv_heads, a.max_ctx, seg.num_segments) *
                           static_cast<size_t>(a.num_heads);
    s.so = reinterpret_cast<float *>(take(align256(entries * static_cast<size_t>(a.head_dim) * 4)));
    s.sml = reinterpret_cast<float2 *>(take(align256(entries * 8)));
    const int64_t pairs = static_cast<int64_t>(a.num_rows) * a.num_heads;
    if (a.fp8) {
        s.q_terms = take(align256(static_cast<size_t>(pairs) * 2 * static_cast<size_t>(a.head_dim)));
        s.q_factor = reinterpret_cast<float *>(take(align256(static_cast<size_t>(pairs) * 4)));
    }
    s.a = a;
    cudaError_t e;
    // nothing to gain in any segment of such a call
    const int64_t most = (a.num_rows / a.group - 1ll) * a.max_ctx * token_bytes(a);
    if (most < least) {
        e = launch_kv_attention(a, workspace, stream);
        if (e != cudaSuccess || a.status == nullptr) return e;
        return launch_pdl(kv_segments_check_kernel, dim3(1), dim3(kSegThreads), 0, stream, s);
    }
    const int64_t at_once = kSegThreads * 16 / a.head_dim;  // queries of a CTA
    const int64_t ctas = a.fp8 ? (pairs + at_once - 1) / at_once : 0;
    e = launch_pdl(kv_segments_kernel, dim3(static_cast<unsigned>(1 + (ctas < kSharedCtas - 1 ? ctas : kSharedCtas - 1))),
                   dim3(kSegThreads), 0, stream, s);
    if (e != cudaSuccess) return e;
    a.row_ctx = s.own_ctx;
    a.row_begin = s.row_begin;
    a.keep_parts = true;
    a.own_sms = s.own_sms;
    e = launch_kv_attention_parts(a, workspace, stream);
    if (e != cudaSuccess) return e;
    s.a = a;
    if (a.fp8) e = a.head_dim == 64 ? launch_shared<true, 64>(s, stream) : launch_shared<true, 128>(s, stream);
    else e = a.head_dim == 64 ? launch_shared<false, 64>(s, stream) : launch_shared<false, 128>(s, stream);
    if (e != cudaSuccess) return e;
    return a.head_dim == 64 ? launch_join<64>(s, stream) : launch_join<128>(s, stream);
}

}  // namespace dsa
