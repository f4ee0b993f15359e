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
// Both kernels move each byte once and do little with it: they are bound by the memory, and by latency for the
// few tokens of a decode step.  One CTA takes a tile of tokens of one tensor (or a range of one token's heads):
// it computes the tile's cos and sin once per (token, pair) into shared memory; then every thread keeps one
// 16-byte piece of a head and walks over the tile's heads and tokens with it, so that the walk has no division and
// the angles' place changes with the token alone.  What it takes is bytes in flight: a thread's next pieces come by
// asynchronous copies into 128 bytes of its own in shared memory (with four 16-byte loads in registers instead, the
// prefills below took 43 and 64.5 us; a ring of 96 bytes 35.2 and 56.5 us).
// 8,192 tokens x 98 heads x 64 dims: 35.8 us (5.7 TB/s; in fp32, 96 heads, 60.9 us, 6.6 TB/s); 8,192 tokens into an
// FP8 pool of 4 KV heads of 128 with 64 query heads rotated: 48.0 us (6.1 TB/s; bf16 pool 48.6 us, 6.2 TB/s).  Rows that
// 16-byte accesses do not fit go element by element: the same rope from an odd element on 158 us, the same insert with
// 90 rotary dims 246 us; a decode step's few tokens take as long as aligned ones (8 tokens: 1.7 and 1.9 us).
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "kernels.h"
#include "ptx.cuh"

namespace dsa {

namespace {

constexpr int kThreads = 128;
constexpr int kTileTokens = 64;                               // most tokens of a tile
constexpr int kTabPairs = 2048;                               // (token, pair) entries of a tile's table
constexpr int kRingBytes = 128;                               // of a thread: its pieces in flight
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

// A thread's way over a tile of nt tokens x nh heads of `units` pieces: always the same piece of a head, the
// heads (and tokens) a CTA's width apart.
struct Walk {
    int unit, tok, h;           // where it stands
    int h0, h_step, tok_step;

    __device__ __forceinline__ Walk(int units, int nt, int nh) {
        const int lanes = kThreads / units, lane = static_cast<int>(threadIdx.x) / units;
        unit = static_cast<int>(threadIdx.x) - lane * units;
        if (nh >= lanes) {
            h0 = lane;
            h_step = lanes;
            tok = 0;
            tok_step = 1;
        } else {
            tok = lane / nh;
            h0 = lane - tok * nh;
            h_step = nh;
            tok_step = lanes / nh;
            if (tok >= tok_step) tok = nt;
        }
        if (lane >= lanes) tok = nt;
        h = h0;
    }
    __device__ __forceinline__ void step(int nh) {
        h += h_step;
        if (h >= nh) {
            h = h0;
            tok += tok_step;
        }
    }
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

// cos and sin of the tile's tokens, times the scale: [token in tile][pair].
struct Table {
    alignas(16) float cos[kTabPairs], sin[kTabPairs];
};

// A token's position as far as its sign goes: negative if one of its axes' is.
template <bool kAxes>
__device__ __forceinline__ int32_t sign_position(const RopeArgs &a, int token) {
    int32_t pos = a.positions[token];
    if constexpr (kAxes)
        for (int x = 1; x < a.num_axes; ++x) pos |= a.positions[x * a.axis_stride + token];
    return pos;
}

// pos_s: the tile's positions (their signs).  kAxes: pair p's angle goes by the position on its own axis; the axes
// of all pairs come with the launch, two bits each.
template <bool kAxes>
__device__ __forceinline__ void fill_table(const RopeArgs &a, Table &tab, int32_t *pos_s, int t0, int nt) {
    const int pairs = a.rot >> 1;
    if (static_cast<int>(threadIdx.x) < nt) pos_s[threadIdx.x] = sign_position<kAxes>(a, t0 + threadIdx.x);
    for (int i = threadIdx.x; i < nt * pairs; i += kThreads) {
        const int tok = i / pairs, p = i - tok * pairs;
        const int32_t *of = a.positions;
        if constexpr (kAxes) of += (a.axis[p >> 4] >> 2 * (p & 15) & 3u) * a.axis_stride;
        const int64_t pos = of[t0 + tok];
        const uint64_t phase = static_cast<uint64_t>(pos) * a.turns[p];
        const float half_turns = static_cast<float>(static_cast<int32_t>(phase >> 32)) * 0x1p-31f;
        float sn, cs;
        sincospif(half_turns, &sn, &cs);
        tab.cos[i] = cs * a.scale;
        tab.sin[i] = sn * a.scale;
    }
}

// N angles from a multiple of N floats.
template <int N>
__device__ __forceinline__ void load_angles(const float *p, float (&v)[N]) {
    if constexpr (N % 4 == 0) {
#pragma unroll
        for (int i = 0; i < N; i += 4) *reinterpret_cast<float4 *>(v + i) = *reinterpret_cast<const float4 *>(p + i);
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = p[i];
    }
}

// (u, v) becomes (u c - v s, u s + v c): two pairs at a time in packed fp32 where there are two.
template <int N>
__device__ __forceinline__ void turn(float (&u)[N], float (&v)[N], const float (&c)[N], const float (&s)[N]) {
    if constexpr (N % 2 == 0) {
#pragma unroll
        for (int e = 0; e < N; e += 2) {
            const float2 u2 = make_float2(u[e], u[e + 1]), v2 = make_float2(v[e], v[e + 1]);
            const float2 c2 = make_float2(c[e], c[e + 1]), s2 = make_float2(s[e], s[e + 1]);
            const float2 a = __ffma2_rn(v2, make_float2(-s2.x, -s2.y), __fmul2_rn(u2, c2));
            const float2 b = __ffma2_rn(v2, c2, __fmul2_rn(u2, s2));
            u[e] = a.x;
            u[e + 1] = a.y;
            v[e] = b.x;
            v[e + 1] = b.y;
        }
    } else {
        const float a = fmaf(v[0], -s[0], u[0] * c[0]);
        v[0] = fmaf(v[0], c[0], u[0] * s[0]);
        u[0] = a;
    }
}

// A piece of a head: V elements (V / 2 pairs) of an interleaved one, or V elements of each half of a half-split
// one.  V = 1 (half) and 2 (interleaved) are the forms for any alignment.
template <typename T, bool kHalf, int V>
struct HeadPiece {
    static constexpr int kPairs = kHalf ? V : V / 2;
    static constexpr bool kWide = kHalf || V * sizeof(T) >= 16;
    using P = Piece<T, V>;
    P lo, hi;
    __device__ __forceinline__ void load(const T *p, int pairs) {
        if constexpr (kWide) {
            lo = *reinterpret_cast<const P *>(p);
            if (kHalf) hi = *reinterpret_cast<const P *>(p + pairs);
        } else {
#pragma unroll
            for (int e = 0; e < V; ++e) lo.e[e] = p[e];
        }
    }
    __device__ __forceinline__ void rotate(const float (&c)[kPairs], const float (&s)[kPairs]) {
        float u[kPairs], v[kPairs];
#pragma unroll
        for (int e = 0; e < kPairs; ++e) {
            u[e] = to_f32(lo.e[kHalf ? e : 2 * e]);
            v[e] = to_f32(kHalf ? hi.e[e] : lo.e[2 * e + 1]);
        }
        turn<kPairs>(u, v, c, s);
#pragma unroll
        for (int e = 0; e < kPairs; ++e) {
            lo.e[kHalf ? e : 2 * e] = from_f32<T>(u[e]);
            (kHalf ? hi.e[e] : lo.e[2 * e + 1]) = from_f32<T>(v[e]);
        }
    }
    __device__ __forceinline__ void store(T *p, int pairs) const {
        if constexpr (kWide) {
            *reinterpret_cast<P *>(p) = lo;
            if (kHalf) *reinterpret_cast<P *>(p + pairs) = hi;
        } else {
#pragma unroll
            for (int e = 0; e < V; ++e) p[e] = lo.e[e];
        }
    }
};

// 16 bytes to shared memory while the thread goes on.  Its own wait makes them visible to it.
__device__ __forceinline__ void copy16(void *dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Rotate the tile's pieces.  The 16-byte forms pass through a ring of the thread's own in shared memory, so that
// several are in flight while one is worked on, the first ones while the table is made.
template <bool kAxes, typename T, bool kHalf, int V>
__device__ __forceinline__ void rotate_tile(const RopeArgs &a, const RopeTensor &x, Table &tab, int32_t *pos_s,
                                            uint8_t *ring, int t0, int nt, int h0, int nh, int units) {
    using H = HeadPiece<T, kHalf, V>;
    const int pairs = a.rot >> 1;
    Walk w(units, nt, nh);
    const T *src = static_cast<const T *>(x.x) + t0 * x.x_token + h0 * x.x_head + w.unit * V;
    T *dst = static_cast<T *>(x.out) + t0 * x.out_token + h0 * x.out_head + w.unit * V;
    const int unit = w.unit * H::kPairs;
    if constexpr (V * sizeof(T) < 16) {
        fill_table<kAxes>(a, tab, pos_s, t0, nt);
        __syncthreads();
        for (; w.tok < nt; w.step(nh)) {
            if (pos_s[w.tok] < 0) continue;  // a padding token
            H piece;
            piece.load(src + w.tok * x.x_token + w.h * x.x_head, pairs);
            float c[H::kPairs], s[H::kPairs];
            load_angles<H::kPairs>(tab.cos + w.tok * pairs + unit, c);
            load_angles<H::kPairs>(tab.sin + w.tok * pairs + unit, s);
            piece.rotate(c, s);
            piece.store(dst + w.tok * x.out_token + w.h * x.out_head, pairs);
        }
    } else {
        constexpr int kBytes = kHalf ? 32 : 16, kDepth = kRingBytes / kBytes;
        // the walk's steps in memory, so that a piece's address takes additions alone
        struct Steps {
            int64_t head, token;  // bytes
            uint8_t *at, *row;    // this piece, and the first one of its token
            __device__ __forceinline__ void step(bool same_token) {
                at += head;
                if (!same_token) at = row += token;
            }
        };
        auto steps = [&](const void *base, int64_t token, int64_t head) {
            Steps p{w.h_step * head * static_cast<int64_t>(sizeof(T)), w.tok_step * token * static_cast<int64_t>(sizeof(T)),
                    nullptr, nullptr};
            p.row = static_cast<uint8_t *>(const_cast<void *>(base)) +
                    (w.tok * token + w.h0 * head) * static_cast<int64_t>(sizeof(T));
            p.at = p.row;
            return p;
        };
        Walk ahead = w;
        Steps from = steps(src, x.x_token, x.x_head), to = steps(dst, x.out_token, x.out_head);
        uint8_t *mine = ring + threadIdx.x * 16;
        constexpr int kPlace = kThreads * 16, kHigh = kDepth * kPlace;  // (the second halves lie behind the first)
        int in = 0, out = 0;                                            // places in the ring
        const int other = pairs * static_cast<int>(sizeof(T));
        auto start = [&]() {
            if (ahead.tok < nt) {
                copy16(mine + in, from.at);
                if (kHalf) copy16(mine + in + kHigh, from.at + other);
                const int tok = ahead.tok;
                ahead.step(nh);
                from.step(ahead.tok == tok);
            }
            copy_commit();
            in = in + kPlace == kHigh ? 0 : in + kPlace;
        };
#pragma unroll 1
        for (int i = 0; i < kDepth - 1; ++i) start();
        fill_table<kAxes>(a, tab, pos_s, t0, nt);
        __syncthreads();
        float c[H::kPairs], s[H::kPairs];  // of the token at hand
        int held = -1;
        bool live = false;
#pragma unroll 1
        while (w.tok < nt) {
            start();
            if (w.tok != held) {
                held = w.tok;
                live = pos_s[held] >= 0;  // (a negative position: a padding token)
                load_angles<H::kPairs>(tab.cos + held * pairs + unit, c);
                load_angles<H::kPairs>(tab.sin + held * pairs + unit, s);
            }
            copy_wait<kDepth - 1>();
            H piece;
            piece.lo = *reinterpret_cast<const typename H::P *>(mine + out);
            if (kHalf) piece.hi = *reinterpret_cast<const typename H::P *>(mine + out + kHigh);
            out = out + kPlace == kHigh ? 0 : out + kPlace;
            if (live) {
                piece.rotate(c, s);
                piece.store(reinterpret_cast<T *>(to.at), pairs);
            }
            w.step(nh);
            to.step(w.tok == held);
        }
        copy_wait<0>();
    }
}

template <bool kAxes, typename T>
__device__ __forceinline__ void rope_segment(const RopeArgs &a, const RopeTensor &x, const Segment &g, uint32_t cta,
                                             Table &tab, int32_t *pos_s, uint8_t *ring) {
    const uint32_t tile = cta / g.head_chunks, chunk = cta - tile * g.head_chunks;
    const int t0 = static_cast<int>(tile * g.tokens), h0 = static_cast<int>(chunk * g.heads);
    const int nt = min(static_cast<int>(g.tokens), a.num_tokens - t0), nh = min(static_cast<int>(g.heads), x.heads - h0);
    const int units = static_cast<int>(g.units);
    constexpr int V = 16 / sizeof(T);
    if (x.half) {
        if (x.vec) rotate_tile<kAxes, T, true, V>(a, x, tab, pos_s, ring, t0, nt, h0, nh, units);
        else rotate_tile<kAxes, T, true, 1>(a, x, tab, pos_s, ring, t0, nt, h0, nh, units);
    } else {
        if (x.vec) rotate_tile<kAxes, T, false, V>(a, x, tab, pos_s, ring, t0, nt, h0, nh, units);
        else rotate_tile<kAxes, T, false, 2>(a, x, tab, pos_s, ring, t0, nt, h0, nh, units);
    }
}

__device__ __forceinline__ const Segment &segment_of(const Plan &p, uint32_t cta, int &which) {
    which = 0;
    while (which + 1 < p.n && cta >= p.s[which + 1].first) ++which;
    return p.s[which];
}

template <typename T, bool kAxes>
__global__ void __launch_bounds__(kThreads, 6) rope_kernel(const __grid_constant__ RopeArgs a,
                                                        const __grid_constant__ Plan p) {
    __shared__ Table tab;
    __shared__ __align__(16) uint8_t ring[kThreads * kRingBytes];
    __shared__ int32_t pos_s[kTileTokens];
    pdl_wait();
    pdl_launch_dependents();
    int j;
    const Segment &g = segment_of(p, blockIdx.x, j);
    rope_segment<kAxes, T>(a, a.t[j], g, blockIdx.x - g.first, tab, pos_s, ring);
}

// x / s rounded to nearest for the quotients that matter here, from r = 1 / s rounded to nearest: one correction
// of x r by its exact remainder gives the rounded quotient (Markstein, IBM J. Res. Dev. 34, 1990).  Quotients of
// 2^20 and more (and infinities) saturate whatever their last bit.
__device__ __forceinline__ float quotient(float x, float s, float r) {
    const float q = x * r;
    const float c = copysignf(fmaf(fmaf(-q, s, x), r, q), x);
    return fabsf(q) < 1048576.f ? c : q;
}

// Two fp32 -> two e4m3 codes, round to nearest even, saturating; lo in the low byte.
__device__ __forceinline__ uint32_t e4m3x2_rne(float lo, float hi) {
    return static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E4M3));
}

// The tile's K and V rows (2 * kv_heads per token: K heads, then V heads) into the pool, V elements
// at a time.  A rotated element of a half-split pair reads its partner too (from L1), so that every
// thread writes one contiguous piece.  slot_s: the tile's slots, negative where nothing is written.
template <int V>
__device__ __forceinline__ void insert_tile(const KvInsertArgs &a, const Table &tab, const int32_t *slot_s, int t0,
                                            int nt) {
    using P = Piece<__nv_bfloat16, V>;
    constexpr int kBatch = V == 8 ? 2 : 1;
    const int rot = a.rope.rot, pairs = rot >> 1, D = a.head_dim, rows = 2 * a.kv_heads;
    Walk w(D / V, nt, rows);
    const int e0 = w.unit * V, r0 = e0 - a.rot_offset;
    const bool turned = r0 >= 0 && r0 < rot;              // this piece of a K head is rotated
    const bool low = r0 < pairs;
    const int partner = a.half ? (low ? pairs : -pairs) : (r0 & 1 ? -1 : 1);  // (interleaved: for V = 1 alone)
    const __nv_bfloat16 *k = reinterpret_cast<const __nv_bfloat16 *>(a.k) + t0 * a.k_stride + e0;
    const __nv_bfloat16 *v = reinterpret_cast<const __nv_bfloat16 *>(a.v) + t0 * a.v_stride + e0;
    while (w.tok < nt) {
        P p[kBatch], q[kBatch];
        int tok[kBatch], row[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            tok[i] = w.tok;
            row[i] = w.h;
            if (w.tok < nt && slot_s[w.tok] < 0) tok[i] = nt;
            if (tok[i] < nt) {
                const bool is_v = row[i] >= a.kv_heads;
                const __nv_bfloat16 *x = is_v ? v + tok[i] * a.v_stride + (row[i] - a.kv_heads) * D
                                              : k + tok[i] * a.k_stride + row[i] * D;
                p[i] = *reinterpret_cast<const P *>(x);
                if (turned && !is_v && (a.half || V == 1)) q[i] = *reinterpret_cast<const P *>(x + partner);
            }
            w.step(rows);
        }
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            if (tok[i] >= nt) continue;
            const bool is_v = row[i] >= a.kv_heads;
            const int h = is_v ? row[i] - a.kv_heads : row[i];
            float x[V];
#pragma unroll
            for (int e = 0; e < V; ++e) x[e] = __bfloat162float(p[i].e[e]);
            if (turned && !is_v) {
                const float *cos = tab.cos + tok[i] * pairs, *sin = tab.sin + tok[i] * pairs;
                if (a.half) {
                    const int first = low ? r0 : r0 - pairs;
                    float c[V], n[V];
                    load_angles<V>(cos + first, c);
                    load_angles<V>(sin + first, n);
#pragma unroll
                    for (int e = 0; e < V; ++e)  // (as turn rounds it)
                        x[e] = low ? fmaf(__bfloat162float(q[i].e[e]), -n[e], x[e] * c[e])
                                   : fmaf(x[e], c[e], __bfloat162float(q[i].e[e]) * n[e]);
                } else if constexpr (V > 1) {
                    float c[V / 2], n[V / 2], u[V / 2], y[V / 2];
                    load_angles<V / 2>(cos + (r0 >> 1), c);
                    load_angles<V / 2>(sin + (r0 >> 1), n);
#pragma unroll
                    for (int e = 0; e < V / 2; ++e) {
                        u[e] = x[2 * e];
                        y[e] = x[2 * e + 1];
                    }
                    turn<V / 2>(u, y, c, n);
#pragma unroll
                    for (int e = 0; e < V / 2; ++e) {
                        x[2 * e] = u[e];
                        x[2 * e + 1] = y[e];
                    }
                } else {
                    const float c = cos[r0 >> 1], n = sin[r0 >> 1], y = __bfloat162float(q[i].e[0]);
                    x[0] = r0 & 1 ? fmaf(x[0], c, y * n) : fmaf(y, -n, x[0] * c);
                }
            }
            const int32_t slot = slot_s[tok[i]];
            const int64_t page = slot >> a.page_shift;
            const int in_page = slot & (a.page_size - 1);
            const int64_t at = (((page * a.kv_heads + h) * 2 + (is_v ? 1 : 0)) * a.page_size + in_page) * D + e0;
            if (a.fp8) {
                const float s = is_v ? a.v_scale : a.k_scale, r = is_v ? a.v_inv : a.k_inv;
                float y[V];
#pragma unroll
                for (int e = 0; e < V; ++e) y[e] = r > 0.f ? quotient(x[e], s, r) : x[e] / s;
                if constexpr (V == 8) {
                    uint2 o;
                    o.x = e4m3x2_rne(y[0], y[1]) | e4m3x2_rne(y[2], y[3]) << 16;
                    o.y = e4m3x2_rne(y[4], y[5]) | e4m3x2_rne(y[6], y[7]) << 16;
                    *reinterpret_cast<uint2 *>(a.pool + at) = o;
                } else {
                    a.pool[at] = static_cast<uint8_t>(e4m3x2_rne(y[0], 0.f));
                }
            } else {
                P o;
#pragma unroll
                for (int e = 0; e < V; ++e) o.e[e] = __float2bfloat16_rn(x[e]);
                *reinterpret_cast<P *>(reinterpret_cast<__nv_bfloat16 *>(a.pool) + at) = o;
            }
        }
    }
}

// Segment 0: the K and V rows; segment 1, if any: q.
template <bool kAxes>
__global__ void __launch_bounds__(kThreads, 6) kv_insert_kernel(const __grid_constant__ KvInsertArgs a,
                                                             const __grid_constant__ Plan p) {
    __shared__ Table tab;
    __shared__ __align__(16) uint8_t ring[kThreads * kRingBytes];
    __shared__ int32_t pos_s[kTileTokens];
    pdl_wait();
    pdl_launch_dependents();
    int j;
    const Segment &g = segment_of(p, blockIdx.x, j);
    const uint32_t cta = blockIdx.x - g.first;
    if (j == 1) {
        rope_segment<kAxes, __nv_bfloat16>(a.rope, a.rope.t[0], g, cta, tab, pos_s, ring);
        return;
    }
    const int t0 = static_cast<int>(cta * g.tokens);
    const int nt = min(static_cast<int>(g.tokens), a.rope.num_tokens - t0);
    __shared__ int32_t slot_s[kTileTokens];
    if (static_cast<int>(threadIdx.x) < nt) {
        int32_t slot = a.slots[t0 + threadIdx.x];
        if (slot >= a.num_slots || (slot >= 0 && a.rope.rot > 0 && sign_position<kAxes>(a.rope, t0 + threadIdx.x) < 0)) {
            report(a.status, DSA_ERR_BOUNDS);
            slot = -1;
        }
        slot_s[threadIdx.x] = slot;
    }
    if (a.rope.rot > 0) fill_table<kAxes>(a.rope, tab, pos_s, t0, nt);
    __syncthreads();
    if (a.vec) insert_tile<8>(a, tab, slot_s, t0, nt);
    else insert_tile<1>(a, tab, slot_s, t0, nt);
}

// Tiles of sixteen pieces a thread once there are enough to fill the GPU, of one a thread, as many CTAs as
// possible, for the few tokens of a decode step.  The two prefills above with 16, 18 and 24 pieces: rope 35.8,
// 35.4 and 35.5 us, insert 48.0, 48.6 and 54.8 us.  "Enough", in pieces, one / sixteen a thread (us in a graph):
//   rope     98,304 (128 tokens of 98 heads of 64)       3.4 / 4.1    196,608  5.4 / 4.1    786,432  14.8 / 7.5
//   insert's q, K and V at one: 262,144 (512 x 64 heads) 7.0 / 8.1    524,288 12.7 / 10.1
//   K and V  262,144 (2,048 tokens of 8 heads of 128)    7.7 / 13.0   524,288 (4,096 of 4, beside q) 33.1 / 31.7
//            1,048,576 (8,192 of 4, beside q)           65.7 / 47.7   (no ring brings their pieces, so that long
//            tiles on few SMs take longer)
constexpr uint64_t kManyRope = 1u << 17, kManyQ = 1u << 19, kManyKv = 1u << 20;

bool add_segment(Plan &p, uint64_t &ctas, int num_tokens, int heads, uint32_t units, int pairs, bool split_heads,
                 uint64_t many) {
    const uint64_t pieces = static_cast<uint64_t>(num_tokens) * heads * units;
    const uint32_t target = pieces >= many ? 16 * kThreads : kThreads;
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
        if (!add_segment(p, ctas, a.num_tokens, a.t[i].heads, rope_units(a.t[i], a.rot, v), a.rot / 2, true, kManyRope))
            return cudaErrorInvalidConfiguration;
    const bool axes = a.num_axes > 1;
    auto kern = dtype == DSA_DTYPE_BF16 ? (axes ? rope_kernel<__nv_bfloat16, true> : rope_kernel<__nv_bfloat16, false>)
                                        : (axes ? rope_kernel<float, true> : rope_kernel<float, false>);
    return launch_pdl(kern, dim3(static_cast<unsigned>(ctas)), dim3(kThreads), 0, s, a, p);
}

cudaError_t launch_kv_insert(const KvInsertArgs &a, cudaStream_t s) {
    if (a.rope.num_tokens == 0) return cudaSuccess;
    Plan p = {};
    uint64_t ctas = 0;
    if (!add_segment(p, ctas, a.rope.num_tokens, 2 * a.kv_heads, static_cast<uint32_t>(a.head_dim / (a.vec ? 8 : 1)),
                     a.rope.rot / 2, false, kManyKv))
        return cudaErrorInvalidConfiguration;
    if (a.rope.num_tensors > 0 &&
        !add_segment(p, ctas, a.rope.num_tokens, a.rope.t[0].heads, rope_units(a.rope.t[0], a.rope.rot, 8),
                     a.rope.rot / 2, true, kManyQ))
        return cudaErrorInvalidConfiguration;
    return launch_pdl(a.rope.num_axes > 1 ? kv_insert_kernel<true> : kv_insert_kernel<false>,
                      dim3(static_cast<unsigned>(ctas)), dim3(kThreads), 0, s, a, p);
}

}  // namespace dsa
