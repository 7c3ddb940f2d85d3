// Rows between the tokens and the sorted positions of their assignments, with
// the weights applied on the way back, and the gradients of both.  Bytes bound
// all of them (a plain copy moves 6.7 TB/s): 4096 tokens x 8 x 6144 bf16 to the
// experts 77 us (6.5 TB/s), back 73 (6.2); the gradients of the way back of 2048
// tokens 75 (6.4), of the way there of 1001 19.4 (5.7).
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
template <>
struct Vec<2> { using T = uint16_t; };
template <>
struct Vec<1> { using T = uint8_t; };

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
        } else if constexpr (N == 1) {
            uint16_t u;
            if (TYPE == kRowBf16) asm("cvt.rn.bf16.f32 %0, %1;" : "=h"(u) : "f"(f[0]));
            else u = __half_as_ushort(__float2half_rn(f[0]));
            v = u;
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
        f = __ldg(a.sorted + p);
        row = p < __ldg(a.npost);
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
                    if (c + u * lanes < c1) v[u] = __ldg(x + c + u * lanes);
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (c + u * lanes < c1) __stcs(out + c + u * lanes, v[u]);
            }
        } else {
            using E = Elems<TYPE, BYTES>;
            const float w = a.weights == nullptr ? 1.0f : __ldg(a.weights + f);
            const V* y = reinterpret_cast<const V*>(static_cast<const uint8_t*>(a.y) + p * a.ldy);
            for (int c = lane; c < vecs; c += lanes * U) {
                V gv[U], yv[U];
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (c + u * lanes < vecs) gv[u] = __ldg(x + c + u * lanes), yv[u] = __ldcs(y + c + u * lanes);
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

// ------------------------------------------------------------------ back to the tokens

// lanes threads to a token's row and kTokenVecs words to a thread, whose rows of
// up to eight slots are under way together.  The sum goes over the slots in
// ascending order in fp32, from add (or zero), and is rounded once.
constexpr int kTokenThreads = 128;
template <int TYPE, int BYTES, int VECS>
__global__ void __launch_bounds__(kTokenThreads) to_tokens_kernel(const ToTokensArgs a, int lanes, int shift, int vecs,
                                                                  int blocks, int64_t total) {
    using E = Elems<TYPE, BYTES>;
    using V = typename Vec<BYTES>::T;
    pdl_trigger();
    pdl_wait();
    const int tid = threadIdx.x, lane = tid & (lanes - 1), per = kTokenThreads >> shift;
    for (int64_t b = blockIdx.x; b < total; b += gridDim.x) {
        const int64_t mb = blocks == 1 ? b : b / blocks, m = mb * per + (tid >> shift);
        const int c0 = (int)(b - mb * blocks) * lanes * VECS + lane;
        if (m >= a.M || c0 >= vecs) continue;
        float s[VECS][E::N];
#pragma unroll
        for (int k = 0; k < VECS; ++k)
#pragma unroll
            for (int q = 0; q < E::N; ++q) s[k][q] = 0.0f;
        if (a.add != nullptr) {
            // (plain loads: out may be add itself)
            const V* add = reinterpret_cast<const V*>(static_cast<const uint8_t*>(a.add) + m * a.ldadd) + c0;
#pragma unroll
            for (int k = 0; k < VECS; ++k)
                if (c0 + k * lanes < vecs) E::get(add[k * lanes], s[k]);
        }
        const int32_t* pos = a.positions + m * a.topk;
        const float* wts = a.weights + (a.weights != nullptr ? m * a.topk : 0);
        for (int j0 = 0; j0 < a.topk; j0 += 8) {
            V v[8][VECS];
            float w[8];
            int p[8];
            unsigned in = 0u;
            // (one word a thread: all positions, then all rows; more of them, small ones, go slot by slot: rows of 6143
            // 75 us instead of 91)
            if (VECS == 1) {
#pragma unroll
                for (int u = 0; u < 8; ++u) {
                    p[u] = j0 + u < a.topk ? __ldg(pos + j0 + u) : -1;
                    w[u] = a.weights != nullptr && j0 + u < a.topk ? __ldg(wts + j0 + u) : 1.0f;
                }
            }
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                if (VECS > 1) {
                    w[u] = 1.0f;
                    if (j0 + u >= a.topk) continue;
                    p[u] = __ldg(pos + j0 + u);
                    if (a.weights != nullptr) w[u] = __ldg(wts + j0 + u);
                }
                if ((uint64_t)(int64_t)p[u] >= (uint64_t)a.cap) continue;
                in |= 1u << u;
                const V* y = reinterpret_cast<const V*>(static_cast<const uint8_t*>(a.y) + (int64_t)p[u] * a.ldy) + c0;
#pragma unroll
                for (int k = 0; k < VECS; ++k)
                    if (c0 + k * lanes < vecs) v[u][k] = __ldcs(y + k * lanes);
            }
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                if (!(in >> u & 1u)) continue;
#pragma unroll
                for (int k = 0; k < VECS; ++k) {
                    if (c0 + k * lanes >= vecs) continue;
                    float f[E::N];
                    E::get(v[u][k], f);
#pragma unroll
                    for (int q = 0; q < E::N; ++q) s[k][q] = __fmaf_rn(w[u], f[q], s[k][q]);
                }
            }
        }
        V* out = static_cast<V*>(a.out) + m * vecs + c0;
#pragma unroll
        for (int k = 0; k < VECS; ++k)
            if (c0 + k * lanes < vecs) out[k * lanes] = E::put(s[k]);
    }
}

// The same of many tokens with rows of whole 8- or 16-byte words: a CTA takes
// every nth piece of lanes * VECS words; a warp has one token at a time, its
// lanes the slots' positions and weights, which are read one piece ahead.  4096
// x 8 rows of 6144: 73 us, 79 by the kernel above; 64 tokens 3.5 and 3.2, rows
// of 6143 138 and 75.
template <int TYPE, int BYTES, int VECS>
__global__ void __launch_bounds__(kTokenThreads)
    to_tokens_many_kernel(const ToTokensArgs a, int lanes, int shift, int vecs, int blocks, int64_t total) {
    using E = Elems<TYPE, BYTES>;
    using V = typename Vec<BYTES>::T;
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
            q.p = __ldg(a.positions + q.m * a.topk + slot);
            if (a.weights != nullptr) q.w = __ldg(a.weights + q.m * a.topk + slot);
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

cudaError_t device_sms(int* sms) {
    int dev = 0;
    const cudaError_t e = cudaGetDevice(&dev);
    return e != cudaSuccess ? e : cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev);
}

template <int MODE, int TYPE, int BYTES>
cudaError_t launch_experts_v(const ToExpertsArgs& a, cudaStream_t st) {
    const int vecs = (int)((int64_t)a.K * row_elem_bytes(a.type) / BYTES);
    // 8- and 16-byte words: 64 threads a row, four words each (4 KB) in a slab; MODE 1 so of many rows (2048 x 8
    // positions of 6144: 75 us, with 128 threads 80, with 256 94), of few 256 (64 x 8: 6.9 us, with 64 7.4).
    // Smaller words, whose instructions count: whole rows (2048 x 4 rows of 6143: 37 us, in slabs 75).
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

template <int TYPE, int BYTES, int VECS>
cudaError_t launch_tokens_n(const ToTokensArgs& a, int vecs, cudaStream_t st) {
    int lanes = 32;
    while (lanes < kTokenThreads && lanes * VECS < vecs) lanes *= 2;
    const int per = kTokenThreads / lanes, blocks = (vecs + lanes * VECS - 1) / (lanes * VECS);
    const int64_t total = ((int64_t)a.M + per - 1) / per * blocks;
    const int64_t ctas = total < ((int64_t)1 << 30) ? total : ((int64_t)1 << 30);
    return launch_overlapped(to_tokens_kernel<TYPE, BYTES, VECS>, dim3((unsigned)ctas), dim3(kTokenThreads), 0, st, a,
                             lanes, log2_of(lanes), vecs, blocks, total);
}
template <int TYPE, int BYTES>
cudaError_t launch_tokens_v(const ToTokensArgs& a, cudaStream_t st) {
    constexpr int VECS = 2;
    const int vecs = (int)((int64_t)a.K * row_elem_bytes(a.type) / BYTES);
    // two words a thread where that leaves enough CTAs
    if ((int64_t)a.M * vecs < (1 << 18)) return launch_tokens_n<TYPE, BYTES, 1>(a, vecs, st);
    if constexpr (BYTES >= 8) {
        int sms = 0;
        const cudaError_t e = device_sms(&sms);
        if (e != cudaSuccess) return e;
        int lanes = 32;
        while (lanes < kTokenThreads && lanes * VECS < vecs) lanes *= 2;
        const int per = kTokenThreads / lanes, blocks = (vecs + lanes * VECS - 1) / (lanes * VECS);
        const int64_t total = ((int64_t)a.M + per - 1) / per * blocks, most = (int64_t)sms * 4;
        const dim3 grid((unsigned)(total < most ? total : most));
        return launch_overlapped(to_tokens_many_kernel<TYPE, BYTES, VECS>, grid, dim3(kTokenThreads), 0, st, a, lanes,
                                 log2_of(lanes), vecs, blocks, total);
    }
    return launch_tokens_n<TYPE, BYTES, VECS>(a, vecs, st);
}

}  // namespace

cudaError_t launch_to_experts(const ToExpertsArgs& a0, cudaStream_t st) {
    ToExpertsArgs a = a0;
    const int eb = row_elem_bytes(a.type);
    a.ldx *= eb;  // bytes from here on
    a.ldy *= eb;
    uintptr_t bits = reinterpret_cast<uintptr_t>(a.x) | reinterpret_cast<uintptr_t>(a.out) | (uintptr_t)a.ldx |
                     (uintptr_t)((int64_t)a.K * eb);
    if (a.y != nullptr) bits |= reinterpret_cast<uintptr_t>(a.y) | (uintptr_t)a.ldy;
    const int v = vec_bytes(bits, eb);
    if (a.grad_w == nullptr) {
        switch (v) {
            case 16: return launch_experts_v<0, kRowU8, 16>(a, st);
            case 8: return launch_experts_v<0, kRowU8, 8>(a, st);
            case 4: return launch_experts_v<0, kRowU8, 4>(a, st);
            case 2: return launch_experts_v<0, kRowU8, 2>(a, st);
            default: return launch_experts_v<0, kRowU8, 1>(a, st);
        }
    }
#define MR_EXPERTS(T)                                              \
    switch (v) {                                                   \
        case 16: return launch_experts_v<1, T, 16>(a, st);         \
        case 8: return launch_experts_v<1, T, 8>(a, st);           \
        case 4: return launch_experts_v<1, T, 4>(a, st);           \
        default: return launch_experts_v<1, T, T == kRowFp32 ? 4 : 2>(a, st); \
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
    uintptr_t bits = reinterpret_cast<uintptr_t>(a.y) | reinterpret_cast<uintptr_t>(a.out) | (uintptr_t)a.ldy |
                     (uintptr_t)((int64_t)a.K * eb);
    if (a.add != nullptr) bits |= reinterpret_cast<uintptr_t>(a.add) | (uintptr_t)a.ldadd;
    const int v = vec_bytes(bits, eb);
#define MR_TOKENS(T)                                               \
    switch (v) {                                                   \
        case 16: return launch_tokens_v<T, 16>(a, st);             \
        case 8: return launch_tokens_v<T, 8>(a, st);               \
        case 4: return launch_tokens_v<T, 4>(a, st);               \
        default: return launch_tokens_v<T, T == kRowFp32 ? 4 : 2>(a, st); \
    }
    if (a.type == kRowBf16) MR_TOKENS(kRowBf16)
    if (a.type == kRowFp16) MR_TOKENS(kRowFp16)
    MR_TOKENS(kRowFp32)
#undef MR_TOKENS
}

}  // namespace mr
