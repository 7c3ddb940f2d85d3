// Host-side plan and launchers of the residual norm and the FP8 quantiser.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace mr {

// 1024 threads x 8 chunks of 8 elements.  Beyond 32768 a thread's chunks do not fit
// its 64 registers, and some 450 bytes of them are spilled: 1024 x 32768 with FP8
// codes 53 us (4.5 TB/s), x 65536 150 (3.1 TB/s).
constexpr int kNormMaxK = 65536;

struct NormArgs {
    const uint16_t *x, *residual, *g;
    uint16_t *sres, *xn;
    float* rstd;
    uint8_t* q;
    void* scale;
    int64_t ldx, ldr, lds;
    int M, K, gemma, fmt;  // fmt: 0 none, 1 MXFP8, 2 MXFP4, 3 FP8 with scales per 128
    float eps;
};

// Chunks of 8 elements that a thread holds; small: CTAs of at most 256 threads.
struct NormPlan {
    int small, chunks;
};
inline NormPlan norm_plan(int M, int K, int sms) {
    const int vpr = K / 8;
    if (M > 2 * sms && vpr <= 2048) {
        const int c = (vpr + 255) / 256;
        return {1, c <= 4 ? c : c <= 6 ? 6 : 8};
    }
    return {0, vpr <= 1024 ? 1 : vpr <= 2048 ? 2 : vpr <= 4096 ? 4 : 8};
}

cudaError_t launch_add_norm(const NormArgs& a, cudaStream_t st);
cudaError_t launch_fp8_quant(const void* x, int64_t ldx, int M, int K, uint8_t* q, float* scale, cudaStream_t st);

}  // namespace mr
