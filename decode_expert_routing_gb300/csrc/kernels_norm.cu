// The residual's addition with the RMSNorm behind it (mr_add_rms_norm) and the
// FP8 quantiser with one fp32 scale per 128 elements (mr_fp8_quant).
#include "common.cuh"
#include "internal.h"
#include "norm_plan.h"

namespace mr {

// ------------------------------------------------------------------ FP8, scales per 128

constexpr int kFp8Group = 128;

// Codes and scale of 8 consecutive bf16 values (one lane of the 16 lanes that
// hold a group of 128; all 32 lanes of the warp call it together):
//   scale = max(amax / 448, 2^-126),  code = e4m3(x * (1 / scale)),
// every fp32 step rounded to nearest.  At the lower bound 1 / scale is finite
// and the smallest bf16, 2^-133, is 2^-7: no value is lost, and a group of
// zeros needs no case of its own.  A NaN makes the scale NaN (the comparison
// keeps it), an infinity makes it infinite: either way the group's products
// are NaN.
__device__ __forceinline__ uint2 fp8_quant_16th(uint4 v, float* scale) {
    unsigned m = vmax_u16x2(vmax_u16x2(v.x & 0x7FFF7FFFu, v.y & 0x7FFF7FFFu),
                            vmax_u16x2(v.z & 0x7FFF7FFFu, v.w & 0x7FFF7FFFu));
#pragma unroll
    for (int o = 1; o < 16; o <<= 1) m = vmax_u16x2(m, __shfl_xor_sync(kFull, m, o));
    const float amax = __uint_as_float(max(m & 0xFFFFu, m >> 16) << 16);
    float s = __fdiv_rn(amax, 448.0f);
    s = s < 0x1p-126f ? 0x1p-126f : s;
    *scale = s;
    const float inv = __frcp_rn(s);
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

// One warp per 128 chunks of 8 elements (8 groups) of a row, four loads in
// flight per lane.
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
#pragma unroll
        for (int u = 0; u < kFp8Unroll; ++u) {
            const int c = c0 + u * 32;
            float s;
            const uint2 q8 = fp8_quant_16th(v[u], &s);
            if (c >= vpr) continue;
            *reinterpret_cast<uint2*>(q + r * K + c * 8) = q8;
            if ((lane & 15) == 0) scale[r * KB + c / 16] = s;
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
// One CTA per row, the row in registers: C chunks of 8 elements a thread.
//   sres = bf16(x + residual)
//   rstd = 1 / sqrt(mean(sres^2) + eps)
//   xn   = bf16((sres * rstd) * s)      (norm_pair, as the route and mr_norm_apply have it)
// and xn's codes, exactly as the quantisers of this library write them.
//
// rstd is the value of the formula rounded once, but for about one row in
// 10^5: the squares of bf16 numbers are exact in fp32, their sum is kept with
// its rounding errors (Knuth's two-sum, hi + lo), and the division and the
// root are put right by one Newton step in the same arithmetic.  What follows
// rounds to bf16, and a rstd one step off would move some values in 10^4 to
// their other neighbour, and the scale of a group with them; it makes the
// codes those of the formula, whatever the order of the sum.

struct Two {
    float hi, lo;
};
__device__ __forceinline__ Two two_add(Two a, Two b) {  // (lo parts: rounding errors, added plainly)
    const ffloat s = ff_two_sum(a.hi, b.hi);
    return {s.hi, __fadd_rn(__fadd_rn(a.lo, b.lo), s.lo)};
}
__device__ __forceinline__ void two_add_to(Two& a, float b) {
    const ffloat s = ff_two_sum(a.hi, b);
    a.hi = s.hi;
    a.lo = __fadd_rn(a.lo, s.lo);
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
    // one step: r + r (1 - (h + l) r^2) / 2, the bracket from the exact square of r
    const float p = __fmul_rn(r, r), pl = __fmaf_rn(r, r, -p);
    float e = __fmaf_rn(-h, p, 1.0f);
    e = __fmaf_rn(-h, pl, e);
    e = __fmaf_rn(-l, p, e);
    return __fmaf_rn(__fmul_rn(r, 0.5f), e, r);
}

template <int C, int FMT>
__global__ void __launch_bounds__(1024) add_norm_kernel(const NormArgs a) {
    __shared__ float s_hi[32], s_lo[32];
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
        v[i] = c < vpr ? ld_stream_v4(a.x + m * a.ldx + c * 8) : zero;
        r[i] = c < vpr && a.residual != nullptr ? ld_stream_v4(a.residual + m * a.ldr + c * 8) : zero;
    }
#pragma unroll
    for (int i = 0; i < C; ++i) {
        const int c = tid + i * nthr;
        g[i] = c < vpr ? ld_ro_v4(a.g + c * 8) : zero;
    }
    Two sum = {0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < C; ++i) {
        if (a.residual != nullptr) {
            uint32_t* p = &v[i].x;
            const uint32_t* q = &r[i].x;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float lo = __fadd_rn(__uint_as_float(p[j] << 16), __uint_as_float(q[j] << 16));
                const float hi = __fadd_rn(__uint_as_float(p[j] & 0xFFFF0000u), __uint_as_float(q[j] & 0xFFFF0000u));
                asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(p[j]) : "f"(hi), "f"(lo));
            }
        }
        const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float lo = __uint_as_float(w[j] << 16), hi = __uint_as_float(w[j] & 0xFFFF0000u);
            two_add_to(sum, __fmul_rn(lo, lo));
            two_add_to(sum, __fmul_rn(hi, hi));
        }
        const int c = tid + i * nthr;
        if (a.sres != nullptr && c < vpr) *reinterpret_cast<uint4*>(a.sres + m * a.lds + c * 8) = v[i];
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        sum = two_add(sum, Two{__shfl_xor_sync(kFull, sum.hi, o), __shfl_xor_sync(kFull, sum.lo, o)});
    if (nw > 1) {
        if (lane == 0) s_hi[warp] = sum.hi, s_lo[warp] = sum.lo;
        __syncthreads();
        sum = lane < nw ? Two{s_hi[lane], s_lo[lane]} : Two{0.0f, 0.0f};
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            sum = two_add(sum, Two{__shfl_xor_sync(kFull, sum.hi, o), __shfl_xor_sync(kFull, sum.lo, o)});
    }
    const float rstd = norm_rstd(sum, a.K, a.eps);
    if (a.rstd != nullptr && tid == 0) a.rstd[m] = rstd;
    if (FMT == 0 && a.xn == nullptr) return;
#pragma unroll
    for (int i = 0; i < C; ++i) {
        const int c = tid + i * nthr;
        const bool in = c < vpr;
        const uint4 n = in ? norm_chunk(v[i], g[i], rstd, a.gemma != 0) : zero;
        if (a.xn != nullptr && in) *reinterpret_cast<uint4*>(a.xn + m * a.K + c * 8) = n;
        if (FMT == 1) {
            unsigned sb;
            const uint2 q = mx_quant_quad(n, &sb);
            if (in) *reinterpret_cast<uint2*>(a.q + m * a.K + c * 8) = q;
            if (in && (lane & 3) == 0) static_cast<uint8_t*>(a.scale)[m * (a.K / 32) + c / 4] = (uint8_t)sb;
        } else if (FMT == 2) {
            unsigned sb;
            const uint32_t q = mx4_quant_quad(n, &sb);
            if (in) *reinterpret_cast<uint32_t*>(a.q + m * (a.K / 2) + c * 4) = q;
            if (in && (lane & 3) == 0) static_cast<uint8_t*>(a.scale)[m * (a.K / 32) + c / 4] = (uint8_t)sb;
        } else if (FMT == 3) {
            float s;
            const uint2 q = fp8_quant_16th(n, &s);
            if (in) *reinterpret_cast<uint2*>(a.q + m * a.K + c * 8) = q;
            if (in && (lane & 15) == 0)
                static_cast<float*>(a.scale)[m * ((a.K + kFp8Group - 1) / kFp8Group) + c / 16] = s;
        }
    }
}

template <int C>
cudaError_t launch_norm_c(const NormArgs& a, int threads, cudaStream_t st) {
    void (*kernel)(const NormArgs) = a.fmt == 0   ? add_norm_kernel<C, 0>
                                     : a.fmt == 1 ? add_norm_kernel<C, 1>
                                     : a.fmt == 2 ? add_norm_kernel<C, 2>
                                                  : add_norm_kernel<C, 3>;
    return launch_overlapped(kernel, dim3((unsigned)a.M), dim3((unsigned)threads), 0, st, a);
}

cudaError_t launch_add_norm(const NormArgs& a, cudaStream_t st) {
    const int vpr = a.K / 8;
    const int c = norm_chunks(vpr), threads = ((vpr + c - 1) / c + 31) / 32 * 32;
    switch (c) {
        case 1: return launch_norm_c<1>(a, threads, st);
        case 2: return launch_norm_c<2>(a, threads, st);
        case 4: return launch_norm_c<4>(a, threads, st);
        default: return launch_norm_c<8>(a, threads, st);
    }
}

}  // namespace mr
