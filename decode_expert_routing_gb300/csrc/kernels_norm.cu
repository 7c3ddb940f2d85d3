// The residual's addition with the RMSNorm behind it (mr_add_rms_norm) and the
// FP8 quantiser with one fp32 scale per 128 elements (mr_fp8_quant).
#include "common.cuh"
#include "internal.h"
#include "norm_plan.h"

namespace mr {

// ------------------------------------------------------------------ FP8, scales per 128

constexpr int kFp8Group = 128;

// Codes and scale of 8 consecutive bf16 values (one lane of the 16 lanes that
// hold a group of 128; all 32 lanes of the warp call these together):
//   scale = max(amax / 448, 2^-126),  code = e4m3(x * (1 / scale)),
// every fp32 step rounded to nearest.  At the lower bound 1 / scale is finite
// and the smallest bf16, 2^-133, is 2^-7: no value is lost, and a group of
// zeros needs no case of its own.  A NaN or an infinity makes the scale NaN
// (the comparison keeps it), and with it every code and product of the group.
__device__ __forceinline__ float fp8_amax_16th(uint4 v) {
    unsigned m = vmax_u16x2(vmax_u16x2(v.x & 0x7FFF7FFFu, v.y & 0x7FFF7FFFu),
                            vmax_u16x2(v.z & 0x7FFF7FFFu, v.w & 0x7FFF7FFFu));
#pragma unroll
    for (int o = 1; o < 16; o <<= 1) m = vmax_u16x2(m, __shfl_xor_sync(kFull, m, o));
    return __uint_as_float(max(m & 0xFFFFu, m >> 16) << 16);
}
// amax / 448 rounded to nearest: a first quotient with the rounded reciprocal,
// put right by its remainder, which is exact (Markstein, "Computation of
// elementary functions on the IBM RISC System/6000 processor", 1990).
__device__ __forceinline__ float fp8_scale(float amax) {
    constexpr float y = 1.0f / 448.0f;
    const float q = __fmul_rn(amax, y);
    const float s = __fmaf_rn(__fmaf_rn(-q, 448.0f, amax), y, q);
    return s < 0x1p-126f ? 0x1p-126f : s;
}
__device__ __forceinline__ uint2 fp8_codes(uint4 v, float inv) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t out[2] = {0u, 0u};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float lo = __fmul_rn(__uint_as_float(w[i] << 16), inv);
        const float hi = __fmul_rn(__uint_as_float(w[i] & 0xFFFF0000u), inv);
        const __nv_fp8x2_storage_t p = __nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E4M3);
        out[i >> 1] |= (uint32_t)p << (16 * (i & 1));
    }
    return make_uint2(out[0], out[1]);
}
// The scales of C chunks (two groups of 128 each in a warp) and their
// reciprocals: lane 16 h + i has that of half h of chunk i, so that the
// reciprocal is computed once for all of them.
template <int C>
__device__ __forceinline__ void fp8_scales(const float (&amax)[C], float (&scale)[C], float (&inv)[C]) {
    static_assert(C <= 16, "a lane of each half for every chunk");
    const int lane = threadIdx.x & 31;
    float mine = amax[0];
#pragma unroll
    for (int i = 1; i < C; ++i) mine = (lane & 15) == i ? amax[i] : mine;
    const float s = fp8_scale(mine), r = __frcp_rn(s);
#pragma unroll
    for (int i = 0; i < C; ++i) {
        scale[i] = __shfl_sync(kFull, s, (lane & 16) + i);
        inv[i] = __shfl_sync(kFull, r, (lane & 16) + i);
    }
}

// One warp per 128 chunks of 8 elements (8 groups) of a row, four loads in
// flight per lane.  Of many rows bytes bound it: 4096 x 6144 14.8 us, 5.2 TB/s, 77 %
// of a plain copy's rate, x 16384 34.4 (5.9 TB/s, 88 %); of few the launch: 1 row
// 1.6 us, 48 1.8, 1000 5.5.
constexpr int kFp8Threads = 256, kFp8Unroll = 4;
__global__ void __launch_bounds__(kFp8Threads) fp8_quant_kernel(const uint16_t* x, int64_t ldx, int M, int K,
                                                                uint8_t* q, float* scale) {
    pdl_trigger();
    pdl_wait();
    const int lane = threadIdx.x & 31, vpr = K / 8, KB = (K + kFp8Group - 1) / kFp8Group;
    const int tpr = (vpr + 32 * kFp8Unroll - 1) / (32 * kFp8Unroll);
    const int64_t tiles = (int64_t)M * tpr, nw = (int64_t)gridDim.x * (kFp8Threads / 32);
    for (int64_t t = (int64_t)blockIdx.x * (kFp8Threads / 32) + (threadIdx.x >> 5); t < tiles; t += nw) {
        const int64_t r = t / tpr;
        const int c0 = (int)(t - r * tpr) * 32 * kFp8Unroll + lane;
        uint4 v[kFp8Unroll];
#pragma unroll
        for (int u = 0; u < kFp8Unroll; ++u) {
            const int c = c0 + u * 32;
            v[u] = c < vpr ? ld_stream_v4(x + r * ldx + c * 8) : make_uint4(0u, 0u, 0u, 0u);
        }
        float amax[kFp8Unroll], s[kFp8Unroll], inv[kFp8Unroll];
#pragma unroll
        for (int u = 0; u < kFp8Unroll; ++u) amax[u] = fp8_amax_16th(v[u]);
        fp8_scales(amax, s, inv);
#pragma unroll
        for (int u = 0; u < kFp8Unroll; ++u) {
            const int c = c0 + u * 32;
            const uint2 q8 = fp8_codes(v[u], inv[u]);
            if (c >= vpr) continue;
            *reinterpret_cast<uint2*>(q + r * K + c * 8) = q8;
            if ((lane & 15) == 0) scale[r * KB + c / 16] = s[u];
        }
    }
}

cudaError_t launch_fp8_quant(const void* x, int64_t ldx, int M, int K, uint8_t* q, float* scale, cudaStream_t st) {
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    const int64_t tiles = (int64_t)M * ((K / 8 + 32 * kFp8Unroll - 1) / (32 * kFp8Unroll));
    int64_t ctas = (tiles + kFp8Threads / 32 - 1) / (kFp8Threads / 32);
    if (ctas > (int64_t)sms * 8) ctas = (int64_t)sms * 8;  // 8 resident CTAs per SM
    return launch_overlapped(fp8_quant_kernel, dim3((unsigned)ctas), dim3(kFp8Threads), 0, st,
                             static_cast<const uint16_t*>(x), ldx, M, K, q, scale);
}

// ------------------------------------------------------------------ residual + RMSNorm
//
// One CTA per row, the row in registers: C chunks of 8 elements a thread.  Of
// many rows memory bounds it: 4096 x 6144 with sres and FP8 codes 34.8 us, 5.1 TB/s,
// 76 % of a plain copy's rate (a row's CTA reads nothing while it sums; persistent
// CTAs that load the next row ahead took 41).  Of few the launch, one load's way
// and the sum's: 1 row 2.5 us, 48 3.1 with MXFP8.
//   sres = bf16(x + residual)
//   rstd = 1 / sqrt(mean(sres^2) + eps)
//   xn   = bf16((sres * rstd) * s)      (norm_pair, as the route and mr_norm_apply have it)
// and xn's codes, exactly as the quantisers of this library write them.
//
// rstd is the value of the formula rounded once, but for about one row in
// 10^5: the squares of bf16 numbers are exact in fp32 (those below 2^-126 but
// for 2^-150), their sum is kept with its rounding errors (Knuth's two-sum, hi
// + lo), and the division and the root are put right by one Newton step in the
// same arithmetic.  What follows rounds to bf16, and a rstd one step off would
// move some values in 10^4 to their other neighbour, and the scale of a group
// with them; it makes the codes those of the formula, whatever the order of the
// sum.  A sum beyond fp32, or one so small that the squares' last bits count
// beside eps, is taken again with scaled squares (norm_again).

struct Two {
    float hi, lo;
};
__device__ __forceinline__ Two two_add(Two a, Two b) {  // (lo parts: rounding errors, added plainly)
    const ffloat s = ff_two_sum(a.hi, b.hi);
    return {s.hi, __fadd_rn(__fadd_rn(a.lo, b.lo), s.lo)};
}
// Two fp32 numbers in one register pair: one instruction for both, each rounded
// by itself.  (At 4096 x 6144 the kernel issued 46 instructions an element, 78 %
// of what the SMs can, and took 38 us.)
typedef unsigned long long Pair;
__device__ __forceinline__ Pair pair_of(uint32_t lo, uint32_t hi) {
    Pair r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(lo), "r"(hi));
    return r;
}
__device__ __forceinline__ void pair_split(Pair p, float& lo, float& hi) {
    uint32_t a, b;
    asm("mov.b64 {%0, %1}, %2;" : "=r"(a), "=r"(b) : "l"(p));
    lo = __uint_as_float(a), hi = __uint_as_float(b);
}
__device__ __forceinline__ Pair pair_add(Pair a, Pair b) {
    Pair r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ Pair pair_sub(Pair a, Pair b) {
    Pair r;
    asm("sub.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ Pair pair_mul(Pair a, Pair b) {
    Pair r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ Pair pair_bf16(uint32_t two) { return pair_of(two << 16, two & 0xFFFF0000u); }
__device__ __forceinline__ uint32_t pair_to_bf16(Pair p) {
    float lo, hi;
    pair_split(p, lo, hi);
    uint32_t d;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
    return d;
}

// Whether a row's sum of squares, taken as they are, is right to 2^-70 of itself
// or of K eps: up to 65536 squares that are each off by at most 2^-150, and
// none of whose sums is beyond fp32 (then it is infinite or NaN).
__device__ __forceinline__ bool norm_fits(Two sum, float eps) {
    return sum.hi < __int_as_float(0x7f800000) && (sum.hi >= 0x1p-60f || eps >= 0x1p-60f);
}
// 1 / sqrt((hi + lo) / K + eps)
__device__ __forceinline__ float norm_rstd(Two sum, int K, float eps) {
    const float k = (float)K;  // exact: K <= 65536
    const float q = __fdiv_rn(sum.hi, k);
    // (hi - q k is exact)
    const float ql = __fdiv_rn(__fadd_rn(__fmaf_rn(-q, k, sum.hi), sum.lo), k);
    const ffloat v = ff_two_sum(q, eps);
    const float h = v.hi, l = __fadd_rn(v.lo, ql);
    const float r = rsqrtf(h);
    if (!(h > 0.0f && h < __int_as_float(0x7f800000))) return r;  // 0, infinite or NaN
    // one step: r + r (1 - (h + l) r r) / 2, the bracket from the exact product h r (the square of r leaves fp32 where
    // h is below 2^-128 or its last bits where h is above 2^100)
    const float t = __fmul_rn(h, r), tl = __fmaf_rn(h, r, -t);
    float e = __fmaf_rn(-t, r, 1.0f);
    e = __fmaf_rn(-tl, r, e);
    e = __fmaf_rn(-__fmul_rn(l, r), r, e);
    return __fmaf_rn(__fmul_rn(r, 0.5f), e, r);
}

// xn and its codes of the chunks c0, c0 + step, ... below vpr of a row m, one
// thread's (a warp's threads call it together); v: the row's values.
template <int C, int FMT>
__device__ __forceinline__ void norm_write(const NormArgs& a, int64_t m, int c0, int step, int vpr, const uint4 (&v)[C],
                                           const uint4 (&g)[C], float rstd) {
    const int lane = threadIdx.x & 31;
    const Pair rr = pair_of(__float_as_uint(rstd), __float_as_uint(rstd)), ones = pair_of(0x3F800000u, 0x3F800000u);
    uint4 n[C];
#pragma unroll
    for (int i = 0; i < C; ++i) {
        // norm_pair's steps (a row's end: zeros, whatever rstd is)
        const int c = c0 + i * step;
        const uint32_t x[4] = {v[i].x, v[i].y, v[i].z, v[i].w}, w[4] = {g[i].x, g[i].y, g[i].z, g[i].w};
        uint32_t* o = &n[i].x;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const Pair k = a.gemma ? pair_add(ones, pair_bf16(w[j])) : pair_bf16(w[j]);
            o[j] = pair_to_bf16(pair_mul(pair_mul(pair_bf16(x[j]), rr), k));
        }
        if (c >= vpr) n[i] = make_uint4(0u, 0u, 0u, 0u);
        if (a.xn != nullptr && c < vpr) *reinterpret_cast<uint4*>(a.xn + m * a.K + c * 8) = n[i];
    }
    if constexpr (FMT == 3) {
        float amax[C], s[C], inv[C];
#pragma unroll
        for (int i = 0; i < C; ++i) amax[i] = fp8_amax_16th(n[i]);
        fp8_scales(amax, s, inv);
#pragma unroll
        for (int i = 0; i < C; ++i) {
            const int c = c0 + i * step;
            const uint2 q = fp8_codes(n[i], inv[i]);
            if (c >= vpr) continue;
            *reinterpret_cast<uint2*>(a.q + m * a.K + c * 8) = q;
            if ((lane & 15) == 0) static_cast<float*>(a.scale)[m * ((a.K + kFp8Group - 1) / kFp8Group) + c / 16] = s[i];
        }
    }
    if constexpr (FMT == 1 || FMT == 2) {
#pragma unroll
        for (int i = 0; i < C; ++i) {
            const int c = c0 + i * step;
            unsigned sb;
            if (FMT == 1) {
                const uint2 q = mx_quant_quad(n[i], &sb);
                if (c < vpr) *reinterpret_cast<uint2*>(a.q + m * a.K + c * 8) = q;
            } else {
                const uint32_t q = mx4_quant_quad(n[i], &sb);
                if (c < vpr) *reinterpret_cast<uint32_t*>(a.q + m * (a.K / 2) + c * 4) = q;
            }
            if (c < vpr && (lane & 3) == 0) static_cast<uint8_t*>(a.scale)[m * (a.K / 32) + c / 4] = (uint8_t)sb;
        }
    }
}

// A row whose sum does not fit, taken again by its whole CTA; small: its sum is
// below 2^-60.  The values of a small one are taken times 2^90, so that every
// square is above 2^-86 and the sum below 2^120; the squares of a large one times
// 2^-32.  Both are exact, but for squares below 2^-94 beside a sum above 2^127.  A
// square beyond fp32, of values from 2^64 on, stays infinite and makes rstd 0; a
// NaN stays one.
// It is a call behind all else and reads the row again: in the kernel's body, from
// the row's registers, it cost every row ten registers a thread.
template <int FMT>
__device__ __noinline__ void norm_again(const NormArgs& a, bool small, float* s_hi, float* s_lo) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nthr = blockDim.x, nw = nthr >> 5;
    const int vpr = a.K / 8;
    const int64_t m = blockIdx.x;
    const float by = small ? 0x1p90f : 1.0f, by2 = small ? 1.0f : 0x1p-32f;
    // (a thread reads the sum that it wrote itself: sres may be x or residual)
    auto chunk = [&](int c) {
        if (a.sres != nullptr) return *reinterpret_cast<const uint4*>(a.sres + m * a.lds + c * 8);
        uint4 v = *reinterpret_cast<const uint4*>(a.x + m * a.ldx + c * 8);
        if (a.residual != nullptr) {
            const uint4 r = *reinterpret_cast<const uint4*>(a.residual + m * a.ldr + c * 8);
            uint32_t* p = &v.x;
            const uint32_t* q = &r.x;
#pragma unroll
            for (int j = 0; j < 4; ++j) p[j] = pair_to_bf16(pair_add(pair_bf16(p[j]), pair_bf16(q[j])));
        }
        return v;
    };
    Two sum{0.0f, 0.0f};
#pragma unroll 1
    for (int c = tid; c < vpr; c += nthr) {
        const uint4 v = chunk(c);
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float x = __fmul_rn(__uint_as_float(j & 1 ? w[j / 2] & 0xFFFF0000u : w[j / 2] << 16), by);
            sum = two_add(sum, Two{__fmul_rn(__fmul_rn(x, x), by2), 0.0f});
        }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        sum = two_add(sum, Two{__shfl_xor_sync(kFull, sum.hi, o), __shfl_xor_sync(kFull, sum.lo, o)});
    __syncthreads();  // (the first sums have been read)
    if (lane == 0) s_hi[warp] = sum.hi, s_lo[warp] = sum.lo;
    __syncthreads();
    sum = lane < nw ? Two{s_hi[lane], s_lo[lane]} : Two{0.0f, 0.0f};
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        sum = two_add(sum, Two{__shfl_xor_sync(kFull, sum.hi, o), __shfl_xor_sync(kFull, sum.lo, o)});
    const float eps = __fmul_rn(__fmul_rn(__fmul_rn(a.eps, by), by), by2);
    const float rstd = __fmul_rn(norm_rstd(sum, a.K, eps), small ? by : 0x1p-16f);
    if (tid == 0 && a.rstd != nullptr) a.rstd[m] = rstd;
    if (FMT == 0 && a.xn == nullptr) return;
#pragma unroll 1
    for (int c = tid; c - lane < vpr; c += nthr) {
        const uint4 zero = make_uint4(0u, 0u, 0u, 0u), v[1] = {c < vpr ? chunk(c) : zero};
        const uint4 g[1] = {c < vpr ? ld_v4(a.g + c * 8) : zero};
        norm_write<1, FMT>(a, m, c, 0, vpr, v, g, rstd);
    }
}

// 16 bytes of a row, streamed; zeros without p.  By predicate, so that a row's loads
// are issued one behind another (in branches 4096 x 6144 with FP8 codes took 35.7
// us, so 34.8; x 8192 45.9 and 42.0).
__device__ __forceinline__ uint4 ld_row_v4(const void* at, bool p) {
    uint4 r = make_uint4(0u, 0u, 0u, 0u);
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %5, 0;\n\t"
        "@q ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];\n\t}"
        : "+r"(r.x), "+r"(r.y), "+r"(r.z), "+r"(r.w)
        : "l"(at), "r"((uint32_t)p));
    return r;
}

// CTAs of 256 threads that an SM's registers are shared among, by the chunks of
// a thread: as many as hold a row's operands with at most 80 bytes spilled, so
// that one row's loads run beside another's sum.  Left to the compiler 4096 x
// 4096 takes 27.0 us with FP8 codes (so 24.3), 26.5 with MXFP8 (23.7), 24.7 without
// (22.6); x 6144 58.2 (34.8), 36.9 (33.0), 35.2 (31.9); x 8192 66.4 (42.0), 53.7
// (40.6), 42.2 (41.5); x 12288 167 (64.7), 71.2 (63.5), 64.7 (61.0); x 16384 132
// (85.4), 125 (90.3), 116 (82.8).  With three chunks FP8 codes, which take more
// registers, are better off with five (4096 x 6144 34.8 us, four 39.9; 500 rows 7.6
// and 7.2), the others with four (500 x 6144 with MXFP8 6.9 us, five 7.8; 4096 33.0
// and 32.3).
constexpr int norm_ctas(int T, int C, int FMT) {
    return T > 256 ? 1 : C == 1 ? 6 : C == 2 ? 5 : C == 3 ? (FMT == 3 ? 5 : 4) : C == 4 ? 4 : C == 6 ? 3 : 2;
}

template <int C, int FMT, int T>
__global__ void __launch_bounds__(T, norm_ctas(T, C, FMT)) add_norm_kernel(const __grid_constant__ NormArgs a) {
    __shared__ float s_hi[32], s_lo[32], s_rstd;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nthr = blockDim.x, nw = nthr >> 5;
    const int vpr = a.K / 8;
    const int64_t m = blockIdx.x;
    pdl_trigger();
    pdl_wait();
    uint4 v[C], r[C], g[C];
    const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
    for (int i = 0; i < C; ++i) {
        const int c = tid + i * nthr;
        v[i] = ld_row_v4(a.x + m * a.ldx + c * 8, c < vpr);
        r[i] = ld_row_v4(a.residual + m * a.ldr + c * 8, c < vpr && a.residual != nullptr);
    }
#pragma unroll
    for (int i = 0; i < C; ++i) {
        const int c = tid + i * nthr;
        g[i] = c < vpr ? ld_v4(a.g + c * 8) : zero;
    }
    Pair hi = 0ull, lo = 0ull;  // sums of the even and of the odd elements' squares, and their rounding errors
#pragma unroll
    for (int i = 0; i < C; ++i) {
        uint32_t* p = &v[i].x;
        const uint32_t* q = &r[i].x;
        if (a.residual != nullptr) {
#pragma unroll
            for (int j = 0; j < 4; ++j) p[j] = pair_to_bf16(pair_add(pair_bf16(p[j]), pair_bf16(q[j])));
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const Pair x = pair_bf16(p[j]), x2 = pair_mul(x, x), s = pair_add(hi, x2), b = pair_sub(s, hi);
            lo = pair_add(lo, pair_add(pair_sub(hi, pair_sub(s, b)), pair_sub(x2, b)));
            hi = s;
        }
        const int c = tid + i * nthr;
        if (a.sres != nullptr && c < vpr) *reinterpret_cast<uint4*>(a.sres + m * a.lds + c * 8) = v[i];
    }
    Two sum, odd;
    pair_split(hi, sum.hi, odd.hi);
    pair_split(lo, sum.lo, odd.lo);
    sum = two_add(sum, odd);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        sum = two_add(sum, Two{__shfl_xor_sync(kFull, sum.hi, o), __shfl_xor_sync(kFull, sum.lo, o)});
    // (of many rows one warp finishes the sum; of few, where a barrier's latency counts, every warp for itself)
    if (lane == 0) s_hi[warp] = sum.hi, s_lo[warp] = sum.lo;
    __syncthreads();
    float rstd;
    if (T > 256 || warp == 0) {
        sum = lane < nw ? Two{s_hi[lane], s_lo[lane]} : Two{0.0f, 0.0f};
#pragma unroll
        for (int o = T > 256 ? 16 : 4; o > 0; o >>= 1)
            sum = two_add(sum, Two{__shfl_xor_sync(kFull, sum.hi, o), __shfl_xor_sync(kFull, sum.lo, o)});
        // (-1, -2: of a sum that does not fit, small or large)
        rstd = norm_rstd(sum, a.K, a.eps);
        rstd = norm_fits(sum, a.eps) ? rstd : sum.hi < 0x1p-60f ? -1.0f : -2.0f;
        if (tid == 0) {
            s_rstd = rstd;
            if (a.rstd != nullptr) a.rstd[m] = rstd;
        }
    }
    if (T <= 256) {
        __syncthreads();
        rstd = s_rstd;
    }
    // (a row whose sum does not fit is written by norm_again alone)
    const bool fits = rstd >= 0.0f;
    if (FMT != 0 || a.xn != nullptr) norm_write<C, FMT>(a, m, tid, nthr, fits ? vpr : 0, v, g, rstd);
    if (!fits) norm_again<FMT>(a, rstd == -1.0f, s_hi, s_lo);
}

template <int C, int T>
cudaError_t launch_norm_c(const NormArgs& a, cudaStream_t st) {
    void (*kernel)(const NormArgs) = a.fmt == 0   ? add_norm_kernel<C, 0, T>
                                     : a.fmt == 1 ? add_norm_kernel<C, 1, T>
                                     : a.fmt == 2 ? add_norm_kernel<C, 2, T>
                                                  : add_norm_kernel<C, 3, T>;
    const int threads = ((a.K / 8 + C - 1) / C + 31) / 32 * 32;
    return launch_overlapped(kernel, dim3((unsigned)a.M), dim3((unsigned)threads), 0, st, a);
}

cudaError_t launch_add_norm(const NormArgs& a, cudaStream_t st) {
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    const NormPlan p = norm_plan(a.M, a.K, sms);
    switch (p.small * 10 + p.chunks) {
        case 11: return launch_norm_c<1, 256>(a, st);
        case 12: return launch_norm_c<2, 256>(a, st);
        case 13: return launch_norm_c<3, 256>(a, st);
        case 14: return launch_norm_c<4, 256>(a, st);
        case 16: return launch_norm_c<6, 256>(a, st);
        case 18: return launch_norm_c<8, 256>(a, st);
        case 1: return launch_norm_c<1, 1024>(a, st);
        case 2: return launch_norm_c<2, 1024>(a, st);
        case 4: return launch_norm_c<4, 1024>(a, st);
        default: return launch_norm_c<8, 1024>(a, st);
    }
}

}  // namespace mr
