// Product of E4M3 operands with fp32 scales per 128, few rows of x
// (mr_fp8_gemm of a decode step's tokens): the weight is streamed once.
//
// A CTA takes 16 A rows of w and 8 B rows of x.  Its eight warps take the
// blocks of K in turn, each for itself: a warp has stages of its own, copies
// into them what it will multiply (tensor maps, 128-byte swizzle), and no
// barrier is shared with another warp until the sums are added at the end, in
// the warps' order.
//
// For a block of 128 a lane reads 32 consecutive bytes of a row of w and of x
// (the swizzle spreads eight lanes over all banks), converts them to f16, which
// every E4M3 value is, and uses each four as the operands of one mma.sync step:
// which of the block's products a step adds is the same permutation of k for
// both operands, and the sum does not depend on it.  (mma.sync on E4M3 itself
// converts both operands again for every step here: 64 rows of x took 33 us with
// 6144 x 6144, 12 without the products.)
//
// The weight's bytes bound it, and for small ones the start: 1 x 6144 x 6144 7.9
// us (4.8 TB/s, with the start's 2; the tensor core kernel took 13.1), 1 x 1536 x
// 6144 5.0, 8 x 6144 x 768 2.8.  The conversions, three cycles each, are why few
// means 16: 16 x 6144 x 6144 9.3 us, 24 by the other kernel 10.9.
#include "../../include/moe_route.h"
#include "fp8_plan.h"
#include "internal.h"
#include "tc_pipe.cuh"
#include "tensor_map.h"

namespace mr {

namespace {

constexpr int kFewWarps = 8;

struct Fp8FewArgs {
    CUtensorMap tm_x, tm_w;  // boxes of 8 B and 16 A rows x 128 bytes
    const float *xs, *ws;
    void* out;
    int64_t ldxs, ldws, ldo;
    unsigned long long wait_ns;
    int M, R, KI, nst, out_fp32, flags;
};

// Four E4M3 values -> two pairs of f16, exactly.
__device__ __forceinline__ uint2 few_f16(uint32_t v) {
    uint2 r;
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
        : "=r"(r.x), "=r"(r.y)
        : "r"(v));
    return r;
}
__device__ __forceinline__ uint4 lds_v4(uint32_t at) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at));
    return v;
}

template <int A, int B>
__global__ void __launch_bounds__(32 * kFewWarps, 2) fp8_few_kernel(const __grid_constant__ Fp8FewArgs a) {
    extern __shared__ __align__(16) unsigned char dsm[];
    __shared__ __align__(8) unsigned long long s_full[kFewWarps][kF8FewStages];
    __shared__ __align__(8) float s_xs[kFewWarps][8 * B];
    __shared__ int s_abort;
    constexpr uint32_t stage = (16 * A + 8 * B) * 128;
    const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(kFull, tid >> 5, 0);
    const int g = lane >> 2, t = lane & 3, r0 = blockIdx.x * (16 * A), m0 = blockIdx.y * (8 * B);
    const uint32_t full = smem_u32(&s_full[warp][0]);
    const uint32_t base = ((smem_u32(dsm) + 1023u) & ~1023u) + (uint32_t)(warp * a.nst) * stage;
    if (lane < kF8FewStages) mbar_init(full + 8u * lane, 1);
    if (tid == 0) {
        s_abort = 0;
        tma_prefetch_map(&a.tm_w);
        tma_prefetch_map(&a.tm_x);
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    // this warp's blocks: warp, warp + 8, ...; its i-th is in stage i % nst
    const int mine = (a.KI - warp + kFewWarps - 1) / kFewWarps;  // (may be negative or 0: none)
    // the weight's way to L2 while the kernel before ends
    if (lane < min(mine, a.nst)) ex_prefetch_2d(&a.tm_w, (warp + lane * kFewWarps) * 128, r0);
    __syncthreads();
    pdl_trigger();
    pdl_wait();

    const uint32_t lead = ex_elect() ? 1u : 0u;
    auto copy = [&](int i, int st) {
        const uint32_t at = base + (uint32_t)st * stage, bar = full + 8u * st;
        const int k = (warp + i * kFewWarps) * 128;
        ex_expect(lead, bar, stage + (((a.flags & 2) && i == 0) ? 16u : 0u));
        ex_load_2d(lead, at, &a.tm_w, k, r0, bar);
        ex_load_2d(lead, at + 16 * A * 128, &a.tm_x, k, m0, bar);
    };
    for (int i = 0; i < min(mine, a.nst); ++i) copy(i, i);

    float acc[A][B][4];
#pragma unroll
    for (int i = 0; i < A; ++i)
#pragma unroll
        for (int n = 0; n < B; ++n)
#pragma unroll
            for (int q = 0; q < 4; ++q) acc[i][n][q] = 0.0f;
    const float* ws = a.ws + (int64_t)(r0 >> 7) * a.ldws;
    float nx = 0.0f, nw = 0.0f;  // of one row of x a lane
    auto fetch = [&](int i) {
        const int kb = warp + i * kFewWarps;
        if (lane < 8 * B && m0 + lane < a.M) nx = a.xs[(int64_t)(m0 + lane) * a.ldxs + kb];
        nw = ws[kb];
    };
    if (mine > 0) fetch(0);
    // bytes of a row's two 16-byte words in a stage: word w of row r is at r * 128 + ((w ^ (r & 7)) << 4)
    const uint32_t o0 = (uint32_t)(g * 128 + (((2 * t) ^ g) << 4)), o1 = (uint32_t)(g * 128 + (((2 * t + 1) ^ g) << 4));
    int st = 0;
    unsigned ph = 0;
    bool ok = true;
    for (int i = 0; i < mine; ++i) {
        // the scales of this block, of w's applied to those of x
        if (lane < 8 * B) s_xs[warp][lane] = __fmul_rn(nx, nw);
        if (i + 1 < mine) fetch(i + 1);
        ok = ex_wait_cta(full + 8u * st, ph, a.wait_ns, &s_abort);  // (and the warp's stores are seen)
        if (!ok) break;
        __syncwarp();
        const uint32_t at = base + (uint32_t)st * stage;
        uint2 w[A][2][8];  // rows g and g + 8, eight times four elements
#pragma unroll
        for (int u = 0; u < A; ++u)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint4 v0 = lds_v4(at + u * 2048u + h * 1024u + o0), v1 = lds_v4(at + u * 2048u + h * 1024u + o1);
                const uint32_t v[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
#pragma unroll
                for (int j = 0; j < 8; ++j) w[u][h][j] = few_f16(v[j]);
            }
#pragma unroll
        for (int n = 0; n < B; ++n) {
            const uint4 v0 = lds_v4(at + 16 * A * 128 + n * 1024u + o0), v1 = lds_v4(at + 16 * A * 128 + n * 1024u + o1);
            const uint32_t v[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
            float p[A][2][4];  // (two chains of steps: one takes some 20 cycles)
#pragma unroll
            for (int u = 0; u < A; ++u)
#pragma unroll
                for (int q = 0; q < 4; ++q) p[u][0][q] = p[u][1][q] = 0.0f;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const uint2 x = few_f16(v[j]);
#pragma unroll
                for (int u = 0; u < A; ++u)
                    mma_f16_m16n8k16(p[u][j & 1], w[u][0][j].x, w[u][1][j].x, w[u][0][j].y, w[u][1][j].y, x.x, x.y);
            }
            const float2 s = *reinterpret_cast<const float2*>(&s_xs[warp][n * 8 + 2 * t]);
#pragma unroll
            for (int u = 0; u < A; ++u)
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    acc[u][n][q] = __fmaf_rn(__fadd_rn(p[u][0][q], p[u][1][q]), (q & 1) ? s.y : s.x, acc[u][n][q]);
        }
        __syncwarp();  // (every lane has read the stage, and the scales)
        if (i + a.nst < mine) copy(i + a.nst, st);
        if (++st == a.nst) st = 0, ph ^= 1u;
    }
    if (!ok && lane == 0) {  // after a wait that ran out: no copy stays in flight (bounded)
        const unsigned long long t0 = global_ns();
        for (int s = 0; s < min(mine, a.nst); ++s)
            while (!mbar_test_cta(full + 8u * s, s >= st ? ph : ph ^ 1u) && global_ns() - t0 < a.wait_ns / 16 + 1000) {
            }
    }
    __syncthreads();
    if (s_abort) return;
    // the warps' sums, [warp][row of x][row of w], where the stages were
    float* sum = reinterpret_cast<float*>(dsm + (((smem_u32(dsm) + 1023u) & ~1023u) - smem_u32(dsm)));
    constexpr int P = 16 * A + 1;
#pragma unroll
    for (int u = 0; u < A; ++u)
#pragma unroll
        for (int n = 0; n < B; ++n)
#pragma unroll
            for (int q = 0; q < 4; ++q)
                sum[(warp * 8 * B + n * 8 + 2 * t + (q & 1)) * P + u * 16 + g + 8 * (q >> 1)] = acc[u][n][q];
    __syncthreads();
    const int rows = min(8 * B, a.M - m0);
    for (int i = tid; i < 16 * A * rows; i += 32 * kFewWarps) {
        const int r = i % (16 * A), m = i / (16 * A);
        if (r0 + r >= a.R) continue;
        float s = 0.0f;
#pragma unroll
        for (int w = 0; w < kFewWarps; ++w) s = __fadd_rn(s, sum[(w * 8 * B + m) * P + r]);
        const int64_t at = (int64_t)(m0 + m) * a.ldo + r0 + r;
        if (a.out_fp32) static_cast<float*>(a.out)[at] = s;
        else static_cast<__nv_bfloat16*>(a.out)[at] = __float2bfloat16_rn(s);
    }
}

template <int A, int B>
cudaError_t launch_few(const Fp8FewArgs& a, const Fp8FewPlan& p, cudaStream_t st) {
    static int prepared[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!__atomic_load_n(&prepared[dev], __ATOMIC_ACQUIRE)) {
        e = cudaFuncSetAttribute(fp8_few_kernel<A, B>, cudaFuncAttributeMaxDynamicSharedMemorySize, kF8FewSmem);
        if (e != cudaSuccess) return e;
        __atomic_store_n(&prepared[dev], 1, __ATOMIC_RELEASE);
    }
    return launch_overlapped(fp8_few_kernel<A, B>, dim3((unsigned)p.gx, (unsigned)p.gy), dim3(32 * kFewWarps),
                             (size_t)p.smem, st, a);
}

}  // namespace

int launch_fp8_few(const Fp8GemmCall& c, int sms, cudaStream_t st, cudaError_t* err) {
    const Fp8FewPlan p = fp8_few_plan(c.M, c.R, c.K, sms);
    Fp8FewArgs a{};
    if (!fp8_encode(&a.tm_x, c.x, c.K, c.M, c.ldx, 8 * p.B) || !fp8_encode(&a.tm_w, c.w, c.K, c.R, c.ldw, 16 * p.A))
        return MR_ERR_UNSUPPORTED;
    a.xs = c.xs;
    a.ws = c.ws;
    a.out = c.out;
    a.ldxs = c.ldxs;
    a.ldws = c.ldws;
    a.ldo = c.ldo;
    a.wait_ns = wait_limit_ns();
    a.M = c.M;
    a.R = c.R;
    a.KI = (c.K + 127) / 128;
    a.nst = p.nst;
    a.out_fp32 = c.out_fp32;
    a.flags = launch_flags();
    switch (p.A * 10 + p.B) {
        case 11: *err = launch_few<1, 1>(a, p, st); break;
        case 12: *err = launch_few<1, 2>(a, p, st); break;
        case 21: *err = launch_few<2, 1>(a, p, st); break;
        default: *err = launch_few<2, 2>(a, p, st); break;
    }
    return *err == cudaSuccess ? MR_OK : MR_ERR_CUDA;
}

int fp8_few_device_error(int clear) {
    int v = 0;
    if (cudaMemcpyFromSymbol(&v, g_ex_timeout, sizeof(int)) != cudaSuccess) return -1;
    if (clear && v) {
        const int z = 0;
        if (cudaMemcpyToSymbol(g_ex_timeout, &z, sizeof(int)) != cudaSuccess) return -1;
    }
    return v;
}

}  // namespace mr
