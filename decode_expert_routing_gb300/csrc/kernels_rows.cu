// Rows between the tokens and the sorted positions of their assignments, with
// the weights applied on the way back, and the gradients of both.  Bytes bound
// all of them (a plain copy moves 6.7 TB/s): 4096 tokens x 8 x 6144 bf16 to the
// experts 77 us (6.5 TB/s), back 72 (6.3); the gradients of the way back of 2048
// tokens 74 (6.4), of the way there of 1001 19.9 (5.6).  (Bytes that a call reads
// and writes; up to 60 MB of what it writes are still in L2 when it ends.)
//
//   mr_moe_permute        rows[p] = x[f / topk]                  f = sorted[p]
//   mr_moe_permute_grad   gx[m]   = sum_j grows[pos[m, j]]
//   mr_moe_combine        out[m]  = add[m] + sum_j w[m, j] y[pos[m, j]]
//   mr_moe_combine_grad   gy[p]   = w[f] gout[f / topk],  gw[f] = <gout[f / topk], y[p]>
//
// The first and the last go by the position (one row is written for each),
// the others by the token: no row has two writers, there are no atomics, and
// every sum has one order.
#include <cuda_fp16.h>

#include "common.cuh"
#include "internal.h"
#include "rows_plan.h"

namespace mr {

namespace {

constexpr int kRowThreads = 256;

template <int BYTES>
struct Vec;
template <>
struct Vec<16> { using T = uint4; };
template <>
struct Vec<8> { using T = uint2; };
template <>
struct Vec<4> { using T = uint32_t; };

// N elements of one vector load as fp32, and back with one rounding.
template <int TYPE, int BYTES>
struct Elems {
    static constexpr int N = BYTES / (TYPE == kRowFp32 ? 4 : 2);
    using V = typename Vec<BYTES>::T;
    static __device__ __forceinline__ void get(const V& v, float (&f)[N]) {
        if constexpr (TYPE == kRowFp32) {
            const uint32_t* w = reinterpret_cast<const uint32_t*>(&v);
#pragma unroll
            for (int i = 0; i < N; ++i) f[i] = __uint_as_float(w[i]);
        } else {
            const uint16_t* w = reinterpret_cast<const uint16_t*>(&v);
#pragma unroll
            for (int i = 0; i < N; ++i)
                f[i] = TYPE == kRowBf16 ? __uint_as_float((uint32_t)w[i] << 16) : __half2float(__ushort_as_half(w[i]));
        }
    }
    static __device__ __forceinline__ V put(const float (&f)[N]) {
        V v;
        if constexpr (TYPE == kRowFp32) {
            uint32_t* w = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
            for (int i = 0; i < N; ++i) w[i] = __float_as_uint(f[i]);
        } else {
            uint32_t* w = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
            for (int i = 0; i < N / 2; ++i) {
                const float a = f[2 * i], b = f[2 * i + 1];
                if (TYPE == kRowBf16) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(b), "f"(a));
                else asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(b), "f"(a));
            }
        }
        return v;
    }
};

// Rows whose words do not start on 16 bytes (odd lengths, odd strides), shifted:
// a thread still takes an aligned 16-byte word of the row that is written, and
// reads the two aligned words that hold those bytes of each other row, which it
// shifts into place.  (Element by element 4096 x 4 rows of 1001 took 27 us each
// way, so 18 and 15.)  Words that leave the operand's memory [lo, hi) are read by
// element, so nothing beside it is.
struct Words {
    uint4 a, b;
    unsigned shift;  // bytes
};
template <int UNIT>
struct Unit;
template <>
struct Unit<1> { using T = uint8_t; };
template <>
struct Unit<2> { using T = uint16_t; };
// A row that is read beside one whose first byte is byte off of its first word: word c of that one are the 16 bytes
// from byte 16 c - off of this one on, those of words [first, last) by aligned words, the others by element.
struct Source {
    const uint8_t* from;  // byte -off
    unsigned shift;
    int first, last;
};
__device__ __forceinline__ Source source(const uint8_t* row, int off, const uint8_t* lo, const uint8_t* hi) {
    Source s;
    s.from = row - off;
    s.shift = (unsigned)(reinterpret_cast<uintptr_t>(s.from) & 15u);
    const uint8_t* g = s.from - s.shift;  // (at most 30 bytes before the row)
    s.first = g >= lo ? 0 : g + 16 >= lo ? 1 : 2;
    const int64_t n = ((hi - g) >> 4) - (s.shift ? 1 : 0);
    s.last = (int)(n < (1 << 30) ? n : (1 << 30));
    return s;
}
// Word c; of one that is read by element the row's bytes [0, end) alone.  UNIT: bytes that every address is a multiple
// of (1 or 2; 4-byte elements by halves).
template <int UNIT>
__device__ __forceinline__ Words load_words(const Source& s, int c, int off, int end) {
    using T = typename Unit<UNIT>::T;
    const uint8_t* from = s.from + (int64_t)c * 16;
    Words r;
    r.shift = s.shift;
    r.b = make_uint4(0u, 0u, 0u, 0u);
    if (c >= s.first && c < s.last) {
        r.a = *reinterpret_cast<const uint4*>(from - s.shift);
        if (s.shift) r.b = *reinterpret_cast<const uint4*>(from - s.shift + 16);
    } else {
        r.shift = 0;
        unsigned long long h0 = 0ull, h1 = 0ull;
#pragma unroll 1
        for (int i = 0; i < 16; i += UNIT) {
            const int at = c * 16 - off + i;
            if (at < 0 || at >= end) continue;
            const unsigned long long e = *reinterpret_cast<const T*>(from + i);
            if (i < 8) h0 |= e << (8 * i);
            else h1 |= e << (8 * i - 64);
        }
        r.a = make_uint4((uint32_t)h0, (uint32_t)(h0 >> 32), (uint32_t)h1, (uint32_t)(h1 >> 32));
    }
    return r;
}
__device__ __forceinline__ uint4 shifted(const Words& v) {
    uint32_t w[8] = {v.a.x, v.a.y, v.a.z, v.a.w, v.b.x, v.b.y, v.b.z, v.b.w};
    const bool two = v.shift & 8u, one = v.shift & 4u;
#pragma unroll
    for (int i = 0; i < 6; ++i) w[i] = two ? w[i + 2] : w[i];
#pragma unroll
    for (int i = 0; i < 5; ++i) w[i] = one ? w[i + 1] : w[i];
    const unsigned bits = (v.shift & 3u) * 8u;
    return make_uint4(__funnelshift_r(w[0], w[1], bits), __funnelshift_r(w[1], w[2], bits),
                      __funnelshift_r(w[2], w[3], bits), __funnelshift_r(w[3], w[4], bits));
}
// The row's bytes among the 16 from byte at on (where they start on 16 bytes of memory).
template <int UNIT>
__device__ __forceinline__ void store_words(uint8_t* row, int at, int end, const uint4& v) {
    using T = typename Unit<UNIT>::T;
    if (at >= 0 && at + 16 <= end) {
        __stcs(reinterpret_cast<uint4*>(row + at), v);
        return;
    }
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 16 / UNIT; ++i)
        if (at + i * UNIT >= 0 && at + i * UNIT < end)
            *reinterpret_cast<T*>(row + at + i * UNIT) = (T)(w[i * UNIT / 4] >> (i * UNIT % 4 * 8));
}

// ------------------------------------------------------------------ to the experts

// lanes threads to a row, kRowThreads / lanes rows to a CTA.  MODE 0: rows as
// they are (any type); 1: weighted, with the weights' gradients.  Padding
// positions give rows of zeros; those behind *npost are left as they are.
// A thread's loads of up to U words are under way together.
//
// MODE 0 goes through the rows in slabs, one slab of every row after the other
// (blockIdx.y): a slab of x stays in L2 for all of its topk reads.  4096 x 8
// rows of 6144, in slabs of 4 KB: 77 us (6.5 TB/s), whole rows 92.  MODE 1 takes
// whole rows, for their sums.
__host__ __device__ constexpr int row_unroll(int bytes) { return bytes >= 8 ? 4 : 6; }
template <int MODE, int TYPE, int BYTES>
__global__ void __launch_bounds__(kRowThreads) to_experts_kernel(const ToExpertsArgs a, int lanes, int shift, int vecs,
                                                                  int slab) {
    using V = typename Vec<BYTES>::T;
    constexpr int U = row_unroll(BYTES);
    __shared__ float s_dot[kRowThreads / 32];
    pdl_trigger();
    pdl_wait();
    const int tid = threadIdx.x, lane = tid & (lanes - 1), mk = a.M * a.topk;
    const int64_t p = ((int64_t)blockIdx.x << (__ffs(kRowThreads) - 1 - shift)) + (tid >> shift);
    int f = -1;
    bool row = false;
    if (p < a.cap) {
        f = a.sorted[p];
        row = p < *a.npost;
    }
    {
        // assignments that the sort left out
        const int64_t i0 = (int64_t)blockIdx.x * kRowThreads + tid;
        if (MODE == 0 && blockIdx.y == 0 && i0 < mk && (unsigned)a.ids[i0] >= (unsigned)a.E) a.positions[i0] = -1;
        if (MODE == 1 && i0 < mk && (uint64_t)(int64_t)a.known[i0] >= (uint64_t)a.cap) a.grad_w[i0] = 0.0f;
    }
    const bool real = row && (unsigned)f < (unsigned)mk;
    V* out = static_cast<V*>(a.out) + p * vecs;
    float dot = 0.0f;
    if (real) {
        const int64_t from = (int64_t)((unsigned)f / (unsigned)a.topk) * a.ldx;
        const V* x = reinterpret_cast<const V*>(static_cast<const uint8_t*>(a.x) + from);
        if constexpr (MODE == 0) {
            if (lane == 0 && blockIdx.y == 0) a.positions[f] = (int32_t)p;
            const int c1 = min((int)(blockIdx.y + 1) * slab, vecs);
            for (int c = (int)blockIdx.y * slab + lane; c < c1; c += lanes * U) {
                V v[U];
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (c + u * lanes < c1) v[u] = x[c + u * lanes];
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (c + u * lanes < c1) __stcs(out + c + u * lanes, v[u]);
            }
        } else {
            using E = Elems<TYPE, BYTES>;
            const float w = a.weights == nullptr ? 1.0f : a.weights[f];
            const V* y = reinterpret_cast<const V*>(static_cast<const uint8_t*>(a.y) + p * a.ldy);
            for (int c = lane; c < vecs; c += lanes * U) {
                V gv[U], yv[U];
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (c + u * lanes < vecs) gv[u] = x[c + u * lanes], yv[u] = __ldcs(y + c + u * lanes);
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    if (c + u * lanes >= vecs) continue;
                    float g[E::N], z[E::N];
                    E::get(gv[u], g);
                    E::get(yv[u], z);
#pragma unroll
                    for (int i = 0; i < E::N; ++i) {
                        dot = __fmaf_rn(g[i], z[i], dot);
                        g[i] = __fmul_rn(w, g[i]);
                    }
                    __stcs(out + c + u * lanes, E::put(g));  // (out may be y itself: its words have been read)
                }
            }
        }
    } else if (row) {
        const int c0 = (int)blockIdx.y * slab, c1 = min(c0 + slab, vecs);
        for (int c = c0 + lane; c < c1; c += lanes) __stcs(out + c, V{});
    }
    if constexpr (MODE == 1) {
        dot = warp_sum_fixed(dot);
        const int warps = lanes / 32, warp = tid >> 5;
        if ((tid & 31) == 0) s_dot[warp] = dot;
        __syncthreads();
        if (real && lane == 0) {
            float s = 0.0f;
            for (int i = 0; i < warps; ++i) s = __fadd_rn(s, s_dot[warp + i]);
            a.grad_w[f] = s;
        }
    }
}

// Rows of 1- and 2-byte units that start anywhere, as they are: to_experts_kernel's MODE 0 with shifted words.  (Rows
// of whole 4- or 8-byte words go faster as such: 2048 x 4 rows of 6142 33 us, shifted 42; of 6143 element by element
// 44, 1000 x 4 30 and 28.)
template <int UNIT>
__global__ void __launch_bounds__(kRowThreads) to_experts_shift_kernel(const ToExpertsArgs a, int lanes, int shift,
                                                                       int slab) {
    constexpr int U = 4;
    pdl_trigger();
    pdl_wait();
    const int tid = threadIdx.x, lane = tid & (lanes - 1), mk = a.M * a.topk;
    const int64_t p = ((int64_t)blockIdx.x << (__ffs(kRowThreads) - 1 - shift)) + (tid >> shift);
    const int64_t i0 = (int64_t)blockIdx.x * kRowThreads + tid;
    if (blockIdx.y == 0 && i0 < mk && (unsigned)a.ids[i0] >= (unsigned)a.E) a.positions[i0] = -1;
    if (p >= a.cap || p >= *a.npost) return;
    const int f = a.sorted[p];
    // the row that is written, its words counted from the 16 bytes that hold its first byte on
    uint8_t* out = static_cast<uint8_t*>(a.out) + p * a.row_bytes;
    const int off = (int)(reinterpret_cast<uintptr_t>(out) & 15u);
    const int c0 = (int)blockIdx.y * slab, c1 = min(c0 + slab, (off + a.row_bytes + 15) / 16);
    if ((unsigned)f >= (unsigned)mk) {
        for (int c = c0 + lane; c < c1; c += lanes)
            store_words<UNIT>(out, c * 16 - off, a.row_bytes, make_uint4(0u, 0u, 0u, 0u));
        return;
    }
    if (lane == 0 && blockIdx.y == 0) a.positions[f] = (int32_t)p;
    const uint8_t* x = static_cast<const uint8_t*>(a.x);
    const Source from = source(x + (int64_t)((unsigned)f / (unsigned)a.topk) * a.ldx, off, x, x + a.x_bytes);
    for (int c = c0 + lane; c < c1; c += lanes * U) {
        Words v[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (c + u * lanes < c1) v[u] = load_words<UNIT>(from, c + u * lanes, off, a.row_bytes);
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (c + u * lanes < c1) store_words<UNIT>(out, (c + u * lanes) * 16 - off, a.row_bytes, shifted(v[u]));
    }
}

// MODE 1 of rows of 2-byte units that start anywhere, both rows shifted.  (2048 x 4 rows of 6143 63 us, element by
// element 67, 16 x 4 4.8 and 8.5; of whole 4- or 8-byte words 63, as such 52 and 49.)
template <int TYPE>
__global__ void __launch_bounds__(kRowThreads) combine_grad_shift_kernel(const ToExpertsArgs a, int lanes, int shift) {
    using E = Elems<TYPE, 16>;
    constexpr int U = 2;
    __shared__ float s_dot[kRowThreads / 32];
    pdl_trigger();
    pdl_wait();
    const int tid = threadIdx.x, lane = tid & (lanes - 1), mk = a.M * a.topk;
    const int64_t p = ((int64_t)blockIdx.x << (__ffs(kRowThreads) - 1 - shift)) + (tid >> shift);
    const int64_t i0 = (int64_t)blockIdx.x * kRowThreads + tid;
    if (i0 < mk && (uint64_t)(int64_t)a.known[i0] >= (uint64_t)a.cap) a.grad_w[i0] = 0.0f;
    int f = -1;
    bool row = false;
    if (p < a.cap) {
        f = a.sorted[p];
        row = p < *a.npost;
    }
    const bool real = row && (unsigned)f < (unsigned)mk;
    // the row that is written, its words counted from the 16 bytes that hold its first byte on
    uint8_t* out = static_cast<uint8_t*>(a.out) + p * a.row_bytes;
    const int off = (int)(reinterpret_cast<uintptr_t>(out) & 15u), words = (off + a.row_bytes + 15) / 16;
    float dot = 0.0f;
    if (real) {
        const uint8_t *x = static_cast<const uint8_t*>(a.x), *y = static_cast<const uint8_t*>(a.y);
        const Source xs = source(x + (int64_t)((unsigned)f / (unsigned)a.topk) * a.ldx, off, x, x + a.x_bytes);
        const Source ys = source(y + p * a.ldy, off, y, y + a.y_bytes);
        const float w = a.weights == nullptr ? 1.0f : a.weights[f];
        for (int c = lane; c < words; c += lanes * U) {
            Words gv[U], yv[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (c + u * lanes >= words) continue;
                gv[u] = load_words<2>(xs, c + u * lanes, off, a.row_bytes);
                yv[u] = load_words<2>(ys, c + u * lanes, off, a.row_bytes);
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (c + u * lanes >= words) continue;
                const int at = (c + u * lanes) * 16 - off;
                float g[E::N], z[E::N];
                E::get(shifted(gv[u]), g);
                E::get(shifted(yv[u]), z);
#pragma unroll
                for (int i = 0; i < E::N; ++i) {
                    if (at + 2 * i >= 0 && at + 2 * i < a.row_bytes) dot = __fmaf_rn(g[i], z[i], dot);
                    g[i] = __fmul_rn(w, g[i]);
                }
                // (out may be y itself: a thread reads its words before it writes them, and no other does)
                store_words<2>(out, at, a.row_bytes, E::put(g));
            }
        }
    } else if (row) {
        for (int c = lane; c < words; c += lanes)
            store_words<2>(out, c * 16 - off, a.row_bytes, make_uint4(0u, 0u, 0u, 0u));
    }
    dot = warp_sum_fixed(dot);
    const int warps = lanes / 32, warp = tid >> 5;
    if ((tid & 31) == 0) s_dot[warp] = dot;
    __syncthreads();
    if (real && lane == 0) {
        float s = 0.0f;
        for (int i = 0; i < warps; ++i) s = __fadd_rn(s, s_dot[warp + i]);
        a.grad_w[f] = s;
    }
}

// ------------------------------------------------------------------ back to the tokens

// lanes threads to a token's row and a word to a thread, whose rows of up to
// eight slots (SHIFT: rows that start anywhere; four) are under way together.
// The sum goes over the slots in ascending order in fp32, from add (or zero), and
// is rounded once.  2048 x 4 rows of 6143: 43 us, element by element 81, of 6140
// 42 and by 8-byte words 46.
constexpr int kTokenThreads = 128;
template <int TYPE, bool SHIFT>
__global__ void __launch_bounds__(kTokenThreads) to_tokens_kernel(const ToTokensArgs a, int lanes, int shift,
                                                                  int blocks, int64_t total) {
    using E = Elems<TYPE, 16>;
    constexpr int U = SHIFT ? 4 : 8;
    pdl_trigger();
    pdl_wait();
    const int tid = threadIdx.x, lane = tid & (lanes - 1), per = kTokenThreads >> shift;
    const uint8_t *y0 = static_cast<const uint8_t*>(a.y), *y1 = y0 + a.y_bytes;
    for (int64_t b = blockIdx.x; b < total; b += gridDim.x) {
        const int64_t mb = blocks == 1 ? b : b / blocks, m = mb * per + (tid >> shift);
        if (m >= a.M) continue;
        // the row that is written, its words counted from the 16 bytes that hold its first byte on
        uint8_t* out = static_cast<uint8_t*>(a.out) + m * a.row_bytes;
        const int off = SHIFT ? (int)(reinterpret_cast<uintptr_t>(out) & 15u) : 0;
        const int c = (int)(b - mb * blocks) * lanes + lane, at = c * 16 - off;
        if (at >= a.row_bytes) continue;
        float s[E::N];
#pragma unroll
        for (int q = 0; q < E::N; ++q) s[q] = 0.0f;
        uint4 start = make_uint4(0u, 0u, 0u, 0u);  // of aligned rows what the sum starts from, waited for with the slots' rows
        if (a.add != nullptr) {
            // (plain loads: out may be add itself)
            const uint8_t *add0 = static_cast<const uint8_t*>(a.add), *add = add0 + m * a.ldadd;
            if (SHIFT) {
                const Source from = source(add, off, add0, add0 + a.add_bytes);
                E::get(shifted(load_words<2>(from, c, off, a.row_bytes)), s);
            } else {
                start = *reinterpret_cast<const uint4*>(add + at);
            }
        }
        const int32_t* pos = a.positions + m * a.topk;
        const float* wts = a.weights + (a.weights != nullptr ? m * a.topk : 0);
        for (int j0 = 0; j0 < a.topk; j0 += U) {
            int p[U];
            float w[U];
            bool in[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                p[u] = j0 + u < a.topk ? pos[j0 + u] : -1;
                w[u] = a.weights != nullptr && j0 + u < a.topk ? wts[j0 + u] : 1.0f;
            }
#pragma unroll
            for (int u = 0; u < U; ++u) in[u] = (uint64_t)(int64_t)p[u] < (uint64_t)a.cap;
            auto add = [&](int u, const uint4& v) {
                float f[E::N];
                E::get(v, f);
#pragma unroll
                for (int q = 0; q < E::N; ++q) s[q] = __fmaf_rn(w[u], f[q], s[q]);
            };
            if constexpr (SHIFT) {
                Words v[U];
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (in[u])
                        v[u] = load_words<2>(source(y0 + (int64_t)p[u] * a.ldy, off, y0, y1), c, off, a.row_bytes);
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (in[u]) add(u, shifted(v[u]));
            } else {
                uint4 v[U];
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (in[u]) v[u] = __ldcs(reinterpret_cast<const uint4*>(y0 + (int64_t)p[u] * a.ldy + at));
                if (j0 == 0) E::get(start, s);
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (in[u]) add(u, v[u]);
            }
        }
        if (SHIFT) store_words<2>(out, at, a.row_bytes, E::put(s));
        else *reinterpret_cast<uint4*>(out + at) = E::put(s);
    }
}

// The same of many tokens with aligned rows: a CTA takes every nth piece of
// lanes * VECS words; a warp has one token at a time, its lanes the slots'
// positions and weights, which are read one piece ahead.  4096 x 8 rows of 6144:
// 73 us, 79 by the kernel above; 64 tokens 3.5 and 3.2.
template <int TYPE, int VECS>
__global__ void __launch_bounds__(kTokenThreads) to_tokens_many_kernel(const ToTokensArgs a, int lanes, int shift,
                                                                       int vecs, int blocks, int64_t total) {
    using E = Elems<TYPE, 16>;
    using V = uint4;
    pdl_trigger();
    pdl_wait();
    const int tid = threadIdx.x, lane = tid & (lanes - 1), slot = tid & 31, per = kTokenThreads >> shift;
    // the piece's token (whole warps agree on it), its first word, and the lane's slot of it
    struct Piece {
        int64_t m;
        int c0, p;
        float w;
    };
    auto fetch = [&](int64_t b) {
        Piece q{a.M, 0, -1, 1.0f};
        if (b >= total) return q;
        const int64_t mb = blocks == 1 ? b : b / blocks;
        q.m = mb * per + (tid >> shift);
        q.c0 = (int)(b - mb * blocks) * lanes * VECS + lane;
        if (q.m < a.M && slot < a.topk) {
            q.p = a.positions[q.m * a.topk + slot];
            if (a.weights != nullptr) q.w = a.weights[q.m * a.topk + slot];
        }
        return q;
    };
    Piece next = fetch(blockIdx.x);
    for (int64_t b = blockIdx.x; b < total; b += gridDim.x) {
        const Piece q = next;
        const bool valid = (uint64_t)(int64_t)q.p < (uint64_t)a.cap;
        const unsigned in = __ballot_sync(kFull, valid);
        const int c0 = q.c0;
        const bool mine = q.m < a.M;
        float s[VECS][E::N];
#pragma unroll
        for (int k = 0; k < VECS; ++k)
#pragma unroll
            for (int i = 0; i < E::N; ++i) s[k][i] = 0.0f;
        V add[VECS];
        if (a.add != nullptr) {
            // (plain loads: out may be add itself)
            const V* from = reinterpret_cast<const V*>(static_cast<const uint8_t*>(a.add) + q.m * a.ldadd) + c0;
#pragma unroll
            for (int k = 0; k < VECS; ++k)
                if (mine && c0 + k * lanes < vecs) add[k] = from[k * lanes];
        }
        for (int j0 = 0; j0 < a.topk; j0 += 8) {
            V v[8][VECS];
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                if (!(in >> (j0 + u) & 1u)) continue;  // (no bit from topk on)
                const int p = __shfl_sync(kFull, q.p, j0 + u);
                const V* y = reinterpret_cast<const V*>(static_cast<const uint8_t*>(a.y) + (int64_t)p * a.ldy) + c0;
#pragma unroll
                for (int k = 0; k < VECS; ++k)
                    if (c0 + k * lanes < vecs) v[u][k] = __ldcs(y + k * lanes);
            }
            if (j0 == 0) {
                next = fetch(b + gridDim.x);
                if (a.add != nullptr) {
#pragma unroll
                    for (int k = 0; k < VECS; ++k)
                        if (mine && c0 + k * lanes < vecs) E::get(add[k], s[k]);
                }
            }
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                if (!(in >> (j0 + u) & 1u)) continue;
                const float w = __shfl_sync(kFull, q.w, j0 + u);
#pragma unroll
                for (int k = 0; k < VECS; ++k) {
                    if (c0 + k * lanes >= vecs) continue;
                    float f[E::N];
                    E::get(v[u][k], f);
#pragma unroll
                    for (int i = 0; i < E::N; ++i) s[k][i] = __fmaf_rn(w, f[i], s[k][i]);
                }
            }
        }
        if (!mine) continue;
        V* out = static_cast<V*>(a.out) + q.m * vecs + c0;
#pragma unroll
        for (int k = 0; k < VECS; ++k)
            if (c0 + k * lanes < vecs) out[k * lanes] = E::put(s[k]);
    }
}

int vec_bytes(uintptr_t bits, int elem) {
    for (int v = 16; v > elem; v >>= 1)
        if ((bits & (uintptr_t)(v - 1)) == 0) return v;
    return elem;
}

int log2_of(int v) {
    int s = 0;
    while ((1 << s) < v) ++s;
    return s;
}

template <int MODE, int TYPE, int BYTES>
cudaError_t launch_experts_v(const ToExpertsArgs& a, cudaStream_t st) {
    const int vecs = a.row_bytes / BYTES;
    // 8- and 16-byte words: 64 threads a row, four words each (4 KB) in a slab; MODE 1 so of many rows (2048 x 8
    // positions of 6144: 75 us, with 128 threads 80, with 256 94), of few 256 (64 x 8: 6.9 us, with 64 7.4).
    // Smaller words, whose instructions count: whole rows (2048 x 4 rows of 6142: 33 us, in slabs twice that).
    const bool wide = BYTES >= 8;
    const int most = !wide ? (MODE == 0 ? 256 : 128) : MODE == 0 || a.cap >= 4096 ? 64 : 256;
    int lanes = 32;
    while (lanes < most && lanes < vecs) lanes *= 2;
    const int64_t per = kRowThreads / lanes, mk = (int64_t)a.M * a.topk;
    int64_t ctas = (a.cap + per - 1) / per;
    if (ctas * kRowThreads < mk) ctas = (mk + kRowThreads - 1) / kRowThreads;  // (a thread for each assignment)
    const int slab = MODE == 0 && wide ? lanes * row_unroll(BYTES) : vecs, slabs = (vecs + slab - 1) / slab;
    const dim3 grid((unsigned)ctas, (unsigned)slabs);
    return launch_overlapped(to_experts_kernel<MODE, TYPE, BYTES>, grid, dim3(kRowThreads), 0, st, a, lanes,
                             log2_of(lanes), vecs, slab);
}

template <int UNIT>
cudaError_t launch_experts_shift(const ToExpertsArgs& a, cudaStream_t st) {
    const int vecs = (a.row_bytes + 30) / 16;  // (at most)
    int lanes = 8;
    while (lanes < 64 && lanes < vecs) lanes *= 2;
    const int64_t per = kRowThreads / lanes, mk = (int64_t)a.M * a.topk;
    int64_t ctas = (a.cap + per - 1) / per;
    if (ctas * kRowThreads < mk) ctas = (mk + kRowThreads - 1) / kRowThreads;  // (a thread for each assignment)
    const int slab = lanes * 4;
    const dim3 grid((unsigned)ctas, (unsigned)((vecs + slab - 1) / slab));
    return launch_overlapped(to_experts_shift_kernel<UNIT>, grid, dim3(kRowThreads), 0, st, a, lanes, log2_of(lanes),
                             slab);
}

template <int TYPE>
cudaError_t launch_combine_grad_shift(const ToExpertsArgs& a, cudaStream_t st) {
    const int vecs = (a.row_bytes + 30) / 16, most = a.cap >= 4096 ? 64 : 256;  // (words: at most; lanes as above)
    int lanes = 32;
    while (lanes < most && lanes < vecs) lanes *= 2;
    const int64_t per = kRowThreads / lanes, mk = (int64_t)a.M * a.topk;
    int64_t ctas = (a.cap + per - 1) / per;
    if (ctas * kRowThreads < mk) ctas = (mk + kRowThreads - 1) / kRowThreads;  // (a thread for each assignment)
    return launch_overlapped(combine_grad_shift_kernel<TYPE>, dim3((unsigned)ctas), dim3(kRowThreads), 0, st, a, lanes,
                             log2_of(lanes));
}

template <int TYPE, bool SHIFT>
cudaError_t launch_tokens_v(const ToTokensArgs& a, cudaStream_t st) {
    const int vecs = (a.row_bytes + (SHIFT ? 15 : 0) + 15) / 16;  // (at most)
    constexpr int VECS = 2;
    if constexpr (!SHIFT) {
        // two words a thread where that leaves enough CTAs
        if ((int64_t)a.M * vecs >= (1 << 18)) {
            int dev = 0, sms = 0;
            cudaError_t e = cudaGetDevice(&dev);
            if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
            if (e != cudaSuccess) return e;
            int lanes = 32;
            while (lanes < kTokenThreads && lanes * VECS < vecs) lanes *= 2;
            const int per = kTokenThreads / lanes, blocks = (vecs + lanes * VECS - 1) / (lanes * VECS);
            const int64_t total = ((int64_t)a.M + per - 1) / per * blocks, most = (int64_t)sms * 4;
            const dim3 grid((unsigned)(total < most ? total : most));
            return launch_overlapped(to_tokens_many_kernel<TYPE, VECS>, grid, dim3(kTokenThreads), 0, st, a, lanes,
                                     log2_of(lanes), vecs, blocks, total);
        }
    }
    int lanes = 8;
    while (lanes < kTokenThreads && lanes < vecs) lanes *= 2;
    const int per = kTokenThreads / lanes, blocks = (vecs + lanes - 1) / lanes;
    const int64_t total = ((int64_t)a.M + per - 1) / per * blocks;
    const int64_t ctas = total < ((int64_t)1 << 30) ? total : ((int64_t)1 << 30);
    return launch_overlapped(to_tokens_kernel<TYPE, SHIFT>, dim3((unsigned)ctas), dim3(kTokenThreads), 0, st, a, lanes,
                             log2_of(lanes), blocks, total);
}
template <int TYPE>
cudaError_t launch_tokens_t(const ToTokensArgs& a, bool aligned, cudaStream_t st) {
    return aligned ? launch_tokens_v<TYPE, false>(a, st) : launch_tokens_v<TYPE, true>(a, st);
}

uintptr_t bits_of(const void* p) { return reinterpret_cast<uintptr_t>(p); }

}  // namespace

cudaError_t launch_to_experts(const ToExpertsArgs& a0, cudaStream_t st) {
    ToExpertsArgs a = a0;
    const int eb = row_elem_bytes(a.type);
    a.ldx *= eb;  // bytes from here on
    a.ldy *= eb;
    a.row_bytes = a.K * eb;
    a.x_bytes = (a.M - 1) * a.ldx + a.row_bytes;
    a.y_bytes = (a.cap - 1) * a.ldy + a.row_bytes;
    uintptr_t bits = bits_of(a.x) | bits_of(a.out) | (uintptr_t)a.ldx | (uintptr_t)a.row_bytes;
    if (a.y != nullptr) bits |= bits_of(a.y) | (uintptr_t)a.ldy;
    const int v = vec_bytes(bits, eb);
    if (a.grad_w == nullptr) {
        switch (v) {
            case 16: return launch_experts_v<0, kRowU8, 16>(a, st);
            case 8: return launch_experts_v<0, kRowU8, 8>(a, st);
            case 4: return launch_experts_v<0, kRowU8, 4>(a, st);
            case 2: return launch_experts_shift<2>(a, st);
            default: return launch_experts_shift<1>(a, st);
        }
    }
    if (v == 2)
        return a.type == kRowBf16 ? launch_combine_grad_shift<kRowBf16>(a, st)
                                  : launch_combine_grad_shift<kRowFp16>(a, st);
#define MR_EXPERTS(T)                                         \
    switch (v) {                                              \
        case 16: return launch_experts_v<1, T, 16>(a, st);    \
        case 8: return launch_experts_v<1, T, 8>(a, st);      \
        default: return launch_experts_v<1, T, 4>(a, st);     \
    }
    if (a.type == kRowBf16) MR_EXPERTS(kRowBf16)
    if (a.type == kRowFp16) MR_EXPERTS(kRowFp16)
    MR_EXPERTS(kRowFp32)
#undef MR_EXPERTS
}

cudaError_t launch_to_tokens(const ToTokensArgs& a0, cudaStream_t st) {
    ToTokensArgs a = a0;
    const int eb = row_elem_bytes(a.type);
    a.ldy *= eb;
    a.ldadd *= eb;
    a.row_bytes = a.K * eb;
    a.y_bytes = (a.cap - 1) * a.ldy + a.row_bytes;
    a.add_bytes = (a.M - 1) * a.ldadd + a.row_bytes;
    uintptr_t bits = bits_of(a.y) | bits_of(a.out) | (uintptr_t)a.ldy | (uintptr_t)a.row_bytes;
    if (a.add != nullptr) bits |= bits_of(a.add) | (uintptr_t)a.ldadd;
    const bool aligned = bits % 16 == 0;
    if (a.type == kRowBf16) return launch_tokens_t<kRowBf16>(a, aligned, st);
    if (a.type == kRowFp16) return launch_tokens_t<kRowFp16>(a, aligned, st);
    return launch_tokens_t<kRowFp32>(a, aligned, st);
}

}  // namespace mr
