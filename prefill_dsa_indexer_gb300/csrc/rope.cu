// rope.cu -- rotary positions (dsa_rope) and the insert of new tokens' keys and values into the
// paged K/V pool (dsa_kv_insert), which rotates K on its way and q beside it.
//
//   out_a = scale (a cos t - b sin t),  out_b = scale (a sin t + b cos t),  t = position * inv_freq_i
//
// Angles.  A position of 10^6 times a frequency in fp32 is off by 2^-24 of 10^6 rad, so the phase is
// kept in turns as 64-bit fixed point: turns_i = inv_freq_i / 2 pi mod 1 in units of 2^-64 turn, and
// position * turns_i mod 2^64 is the phase with its whole turns dropped exactly.  Its top 32 bits, as
// a signed number, are the phase in [-1/2, 1/2) turn; rounding them to fp32 costs at most 2^-26 turn
// (4e-7 rad at half a turn, less nearer 0) at any position.  sincospi then needs no range reduction.
//
// Both kernels move each byte once and do little with it.  One CTA takes a tile of tokens of one
// tensor (or a range of one token's heads): it computes the tile's cos and sin once per (token, pair)
// into shared memory, then every thread rotates 16-byte pieces of the tile's heads, four in flight.
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "kernels.h"
#include "ptx.cuh"

namespace dsa {

namespace {

constexpr int kThreads = 256;
constexpr int kTileTokens = 32;                               // most tokens of a tile
constexpr int kTabPairs = 2048;                               // (token, pair) entries of a tile's table
constexpr int kUnroll = 4;
constexpr int kMaxSegs = DSA_ROPE_MAX_TENSORS + 1;

// A run of CTAs that share one tensor: tiles of `tokens` tokens by `heads` heads.
struct Segment {
    uint32_t first;         // its first CTA
    uint32_t head_chunks;   // CTAs per token tile
    uint32_t tokens, heads; // tile
    uint32_t units;         // pieces per head
};

struct Plan {
    Segment s[kMaxSegs];
    int32_t n;
};

// n / d for n < 2^16, d < 2^16 (m = ceil(2^32 / d), exact in that range; d = 1 has no 32-bit m).
struct Div {
    uint32_t d, m;
    __device__ explicit Div(uint32_t div) : d(div), m(div > 1 ? 0xffffffffu / div + 1 : 0) {}
    __device__ uint32_t quot(uint32_t n) const { return d > 1 ? __umulhi(n, m) : n; }
};

template <typename T>
__device__ __forceinline__ float to_f32(T x);
template <>
__device__ __forceinline__ float to_f32(float x) { return x; }
template <>
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
template <typename T>
__device__ __forceinline__ T from_f32(float x);
template <>
__device__ __forceinline__ float from_f32(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32(float x) { return __float2bfloat16_rn(x); }

template <typename T, int V>
struct alignas(V * sizeof(T)) Piece {
    T e[V];
};

// cos and sin of the tile's tokens, times the scale: tab[token in tile][pair].
__device__ __forceinline__ void fill_table(const RopeArgs &a, float2 *tab, int t0, int nt) {
    const int pairs = a.rot >> 1;
    const Div dv(static_cast<uint32_t>(pairs));
    for (int i = threadIdx.x; i < nt * pairs; i += kThreads) {
        const int tok = static_cast<int>(dv.quot(i)), p = i - tok * pairs;
        const int64_t pos = a.positions[t0 + tok];
        const uint64_t phase = static_cast<uint64_t>(pos) * a.turns[p];
        const float half_turns = static_cast<float>(static_cast<int32_t>(phase >> 32)) * 0x1p-31f;
        float sn, cs;
        sincospif(half_turns, &sn, &cs);
        tab[i] = make_float2(cs * a.scale, sn * a.scale);
    }
}

// Rotate the tile's pieces: V elements (V / 2 pairs) of an interleaved head, or V elements of each
// half of a half-split head.  V = 1 (half) and 2 (interleaved) are the forms for any alignment.
template <typename T, bool kHalf, int V>
__device__ __forceinline__ void rotate_tile(const RopeArgs &a, const RopeTensor &x, const float2 *tab, int t0, int nt,
                                            int h0, int nh, uint32_t units) {
    using P = Piece<T, V>;
    const int pairs = a.rot >> 1;
    const Div du(units), dh(static_cast<uint32_t>(nh));
    const uint32_t total = static_cast<uint32_t>(nt * nh) * units;
    const T *src = static_cast<const T *>(x.x);
    T *dst = static_cast<T *>(x.out);
    for (uint32_t i0 = threadIdx.x; i0 < total; i0 += kThreads * kUnroll) {
        P lo[kUnroll], hi[kUnroll];
        int64_t to[kUnroll];
        int ent[kUnroll];
#pragma unroll
        for (int k = 0; k < kUnroll; ++k) {
            const uint32_t i = i0 + k * kThreads;
            ent[k] = -1;
            if (i >= total) continue;
            const uint32_t row = du.quot(i), u = i - row * units;
            const uint32_t tok = dh.quot(row), h = row - tok * nh;
            if (a.positions[t0 + tok] < 0) continue;
            ent[k] = static_cast<int>(tok) * pairs + static_cast<int>(u) * (kHalf ? V : V / 2);
            const int64_t from = (t0 + static_cast<int64_t>(tok)) * x.x_token + (h0 + static_cast<int64_t>(h)) * x.x_head + u * V;
            to[k] = (t0 + static_cast<int64_t>(tok)) * x.out_token + (h0 + static_cast<int64_t>(h)) * x.out_head + u * V;
            if constexpr (V * sizeof(T) >= 16 || kHalf) {
                lo[k] = *reinterpret_cast<const P *>(src + from);
                if (kHalf) hi[k] = *reinterpret_cast<const P *>(src + from + pairs);
            } else {
#pragma unroll
                for (int e = 0; e < V; ++e) lo[k].e[e] = src[from + e];
            }
        }
#pragma unroll
        for (int k = 0; k < kUnroll; ++k) {
            if (ent[k] < 0) continue;
            const float2 *cs = tab + ent[k];
            if constexpr (kHalf) {
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    const float p = to_f32(lo[k].e[e]), q = to_f32(hi[k].e[e]);
                    lo[k].e[e] = from_f32<T>(p * cs[e].x - q * cs[e].y);
                    hi[k].e[e] = from_f32<T>(p * cs[e].y + q * cs[e].x);
                }
                *reinterpret_cast<P *>(dst + to[k]) = lo[k];
                *reinterpret_cast<P *>(dst + to[k] + pairs) = hi[k];
            } else {
#pragma unroll
                for (int e = 0; e < V / 2; ++e) {
                    const float p = to_f32(lo[k].e[2 * e]), q = to_f32(lo[k].e[2 * e + 1]);
                    lo[k].e[2 * e] = from_f32<T>(p * cs[e].x - q * cs[e].y);
                    lo[k].e[2 * e + 1] = from_f32<T>(p * cs[e].y + q * cs[e].x);
                }
                if constexpr (V * sizeof(T) >= 16) {
                    *reinterpret_cast<P *>(dst + to[k]) = lo[k];
                } else {
#pragma unroll
                    for (int e = 0; e < V; ++e) dst[to[k] + e] = lo[k].e[e];
                }
            }
        }
    }
}

template <typename T>
__device__ __forceinline__ void rope_segment(const RopeArgs &a, const RopeTensor &x, const Segment &g, uint32_t cta,
                                             float2 *tab) {
    const uint32_t tile = cta / g.head_chunks, chunk = cta - tile * g.head_chunks;
    const int t0 = static_cast<int>(tile * g.tokens), h0 = static_cast<int>(chunk * g.heads);
    const int nt = min(static_cast<int>(g.tokens), a.num_tokens - t0), nh = min(static_cast<int>(g.heads), x.heads - h0);
    fill_table(a, tab, t0, nt);
    __syncthreads();
    constexpr int V = 16 / sizeof(T);
    if (x.half) {
        if (x.vec) rotate_tile<T, true, V>(a, x, tab, t0, nt, h0, nh, g.units);
        else rotate_tile<T, true, 1>(a, x, tab, t0, nt, h0, nh, g.units);
    } else {
        if (x.vec) rotate_tile<T, false, V>(a, x, tab, t0, nt, h0, nh, g.units);
        else rotate_tile<T, false, 2>(a, x, tab, t0, nt, h0, nh, g.units);
    }
}

__device__ __forceinline__ const Segment &segment_of(const Plan &p, uint32_t cta, int &which) {
    which = 0;
    while (which + 1 < p.n && cta >= p.s[which + 1].first) ++which;
    return p.s[which];
}

template <typename T>
__global__ void __launch_bounds__(kThreads) rope_kernel(const __grid_constant__ RopeArgs a,
                                                        const __grid_constant__ Plan p) {
    __shared__ __align__(16) float2 tab[kTabPairs];
    pdl_wait();
    pdl_launch_dependents();
    int j;
    const Segment &g = segment_of(p, blockIdx.x, j);
    rope_segment<T>(a, a.t[j], g, blockIdx.x - g.first, tab);
}

__device__ __forceinline__ uint32_t e4m3_rne(float x) {
    return static_cast<uint32_t>(__nv_cvt_float_to_fp8(x, __NV_SATFINITE, __NV_E4M3));
}

// The tile's K and V rows (2 * kv_heads per token: K heads, then V heads) into the pool, V elements
// at a time.  A rotated element of a half-split pair reads its partner too (from L1), so that every
// thread writes one contiguous piece.
template <int V>
__device__ __forceinline__ void insert_tile(const KvInsertArgs &a, const float2 *tab, int t0, int nt) {
    using P = Piece<__nv_bfloat16, V>;
    const int rot = a.rope.rot, pairs = rot >> 1, D = a.head_dim;
    const uint32_t units = static_cast<uint32_t>(D / V), rows = 2 * static_cast<uint32_t>(a.kv_heads);
    const Div du(units), dr(rows);
    const uint32_t total = static_cast<uint32_t>(nt) * rows * units;
    for (uint32_t i = threadIdx.x; i < total; i += kThreads) {
        const uint32_t row = du.quot(i), u = i - row * units;
        const uint32_t tok = dr.quot(row), j = row - tok * rows;
        const int32_t slot = a.slots[t0 + tok];
        if (slot < 0) continue;
        if (slot >= a.num_slots || (rot > 0 && a.rope.positions[t0 + tok] < 0)) {
            if (u == 0 && j == 0) report(a.status, DSA_ERR_BOUNDS);
            continue;
        }
        const bool is_v = j >= static_cast<uint32_t>(a.kv_heads);
        const uint32_t h = is_v ? j - a.kv_heads : j;
        const __nv_bfloat16 *head = reinterpret_cast<const __nv_bfloat16 *>(is_v ? a.v : a.k) +
                                    (t0 + static_cast<int64_t>(tok)) * (is_v ? a.v_stride : a.k_stride) +
                                    static_cast<int64_t>(h) * D;
        const int e0 = static_cast<int>(u) * V;
        float x[V];
        {
            const P p = *reinterpret_cast<const P *>(head + e0);
#pragma unroll
            for (int e = 0; e < V; ++e) x[e] = __bfloat162float(p.e[e]);
        }
        const int r0 = e0 - a.rot_offset;
        if (!is_v && r0 >= 0 && r0 < rot) {
            const float2 *cs = tab + tok * pairs;
            if (a.half) {
                const bool low = r0 < pairs;
                const P p = *reinterpret_cast<const P *>(head + e0 + (low ? pairs : -pairs));
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    const float2 w = cs[(low ? r0 : r0 - pairs) + e];
                    const float y = __bfloat162float(p.e[e]);
                    x[e] = low ? x[e] * w.x - y * w.y : y * w.y + x[e] * w.x;
                }
            } else if constexpr (V > 1) {
#pragma unroll
                for (int e = 0; e < V; e += 2) {
                    const float2 w = cs[(r0 + e) >> 1];
                    const float p = x[e], q = x[e + 1];
                    x[e] = p * w.x - q * w.y;
                    x[e + 1] = p * w.y + q * w.x;
                }
            } else {
                const bool even = (r0 & 1) == 0;
                const float2 w = cs[r0 >> 1];
                const float y = __bfloat162float(head[e0 + (even ? 1 : -1)]);
                x[0] = even ? x[0] * w.x - y * w.y : y * w.y + x[0] * w.x;
            }
        }
        const int64_t page = slot / a.page_size;
        const int in_page = slot % a.page_size;
        const int64_t at = (((page * a.kv_heads + h) * 2 + (is_v ? 1 : 0)) * a.page_size + in_page) * D + e0;
        if (a.fp8) {
            const float s = is_v ? a.v_scale : a.k_scale;  // divided by, not multiplied by its reciprocal
            if constexpr (V == 8) {
                uint2 w;
                w.x = e4m3_rne(x[0] / s) | e4m3_rne(x[1] / s) << 8 | e4m3_rne(x[2] / s) << 16 | e4m3_rne(x[3] / s) << 24;
                w.y = e4m3_rne(x[4] / s) | e4m3_rne(x[5] / s) << 8 | e4m3_rne(x[6] / s) << 16 | e4m3_rne(x[7] / s) << 24;
                *reinterpret_cast<uint2 *>(a.pool + at) = w;
            } else {
                a.pool[at] = static_cast<uint8_t>(e4m3_rne(x[0] / s));
            }
        } else {
            P p;
#pragma unroll
            for (int e = 0; e < V; ++e) p.e[e] = __float2bfloat16_rn(x[e]);
            *reinterpret_cast<P *>(reinterpret_cast<__nv_bfloat16 *>(a.pool) + at) = p;
        }
    }
}

// Segment 0: the K and V rows; segment 1, if any: q.
__global__ void __launch_bounds__(kThreads) kv_insert_kernel(const __grid_constant__ KvInsertArgs a,
                                                             const __grid_constant__ Plan p) {
    __shared__ __align__(16) float2 tab[kTabPairs];
    pdl_wait();
    pdl_launch_dependents();
    int j;
    const Segment &g = segment_of(p, blockIdx.x, j);
    const uint32_t cta = blockIdx.x - g.first;
    if (j == 1) {
        rope_segment<__nv_bfloat16>(a.rope, a.rope.t[0], g, cta, tab);
        return;
    }
    const int t0 = static_cast<int>(cta * g.tokens);
    const int nt = min(static_cast<int>(g.tokens), a.rope.num_tokens - t0);
    if (a.rope.rot > 0) {
        fill_table(a.rope, tab, t0, nt);
        __syncthreads();
    }
    if (a.vec) insert_tile<8>(a, tab, t0, nt);
    else insert_tile<1>(a, tab, t0, nt);
}

// Tiles of about 1,024 pieces (four per thread) once there are enough to fill the GPU, of 256 (one
// per thread, as many CTAs as possible) for the few tokens of a decode step.
bool add_segment(Plan &p, uint64_t &ctas, int num_tokens, int heads, uint32_t units, int pairs, bool split_heads) {
    const uint64_t pieces = static_cast<uint64_t>(num_tokens) * heads * units;
    const uint32_t target = pieces >= (1u << 20) ? kThreads * kUnroll : kThreads;
    Segment &g = p.s[p.n++];
    const uint32_t per_token = static_cast<uint32_t>(heads) * units;
    g.units = units;
    g.first = static_cast<uint32_t>(ctas);
    g.heads = static_cast<uint32_t>(heads);
    g.tokens = 1;
    if (per_token > target && split_heads) {
        g.heads = target / units > 0 ? target / units : 1;
    } else {
        uint32_t t = target / per_token;
        const uint32_t cap = pairs > 0 ? static_cast<uint32_t>(kTabPairs / pairs) : kTileTokens;
        t = t < 1 ? 1 : t;
        t = t > kTileTokens ? kTileTokens : t;
        g.tokens = t > cap ? cap : t;
    }
    g.head_chunks = (static_cast<uint32_t>(heads) + g.heads - 1) / g.heads;
    ctas += (static_cast<uint64_t>(num_tokens) + g.tokens - 1) / g.tokens * g.head_chunks;
    return ctas <= 0x7fffffffull;
}

uint32_t rope_units(const RopeTensor &t, int rot, int vec_elems) {
    if (!t.vec) return static_cast<uint32_t>(rot / 2);
    return static_cast<uint32_t>(t.half ? rot / 2 / vec_elems : rot / vec_elems);
}

}  // namespace

cudaError_t launch_rope(const RopeArgs &a, int32_t dtype, cudaStream_t s) {
    if (a.num_tokens == 0) return cudaSuccess;
    Plan p = {};
    uint64_t ctas = 0;
    const int v = dtype == DSA_DTYPE_BF16 ? 8 : 4;
    for (int i = 0; i < a.num_tensors; ++i)
        if (!add_segment(p, ctas, a.num_tokens, a.t[i].heads, rope_units(a.t[i], a.rot, v), a.rot / 2, true))
            return cudaErrorInvalidConfiguration;
    return dtype == DSA_DTYPE_BF16
               ? launch_pdl(rope_kernel<__nv_bfloat16>, dim3(static_cast<unsigned>(ctas)), dim3(kThreads), 0, s, a, p)
               : launch_pdl(rope_kernel<float>, dim3(static_cast<unsigned>(ctas)), dim3(kThreads), 0, s, a, p);
}

cudaError_t launch_kv_insert(const KvInsertArgs &a, cudaStream_t s) {
    if (a.rope.num_tokens == 0) return cudaSuccess;
    Plan p = {};
    uint64_t ctas = 0;
    if (!add_segment(p, ctas, a.rope.num_tokens, 2 * a.kv_heads, static_cast<uint32_t>(a.head_dim / (a.vec ? 8 : 1)),
                     a.rope.rot / 2, false))
        return cudaErrorInvalidConfiguration;
    if (a.rope.num_tensors > 0 &&
        !add_segment(p, ctas, a.rope.num_tokens, a.rope.t[0].heads, rope_units(a.rope.t[0], a.rope.rot, 8),
                     a.rope.rot / 2, true))
        return cudaErrorInvalidConfiguration;
    return launch_pdl(kv_insert_kernel, dim3(static_cast<unsigned>(ctas)), dim3(kThreads), 0, s, a, p);
}

}  // namespace dsa
