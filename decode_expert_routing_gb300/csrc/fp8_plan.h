// Host-side plan of the FP8 product with scales per 128.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace mr {

struct Fp8GemmCall {
    const uint8_t *x, *w;
    const float *xs, *ws;
    int64_t ldx, ldw, ldxs, ldws, ldo;
    int M, R, K, out_fp32;
    void* out;
};

constexpr int kF8Smem = 208 * 1024;  // dynamic shared memory of a CTA
constexpr int kF8MaxStages = 24;

// Tiles: rows of x are the accumulator's lanes (128 a CTA, 256 a pair), n
// rows of w its columns.
struct Fp8Plan {
    int pair, n, xrows, RT, CT, D, mc, nst, nbuf, grid;  // mc: chunks of 16 columns of a read-back warp
};
inline Fp8Plan fp8_plan(int M, int R, int K, int sms) {
    Fp8Plan p{};
    p.pair = sms >= 2 && M > 128 && (int64_t)((M + 255) / 256) * ((R + 255) / 256) * 2 >= sms;
    const int of = p.pair ? 2 : 1, slots = sms / of;
    p.RT = p.pair ? (M + 255) / 256 : (M + 127) / 128;
    p.xrows = p.pair || M >= 128 ? 128 : (M + 7) / 8 * 8;
    int64_t least = INT64_MAX;
    for (int n = 192; n >= (p.pair ? 64 : 16); n -= 16 * of) {
        const int ct = (R + n - 1) / n;
        const int64_t rounds = ((int64_t)p.RT * ct + slots - 1) / slots;
        const int64_t cost = rounds * (p.pair ? n + 8 : n + p.xrows / 2 + 16);
        if (cost < least) least = cost, p.n = n, p.CT = ct;
    }
    // blocks of a stage: as many as leave two buffers of accumulators and four stages
    const int block = (p.xrows + p.n / of) * 128, room = kF8Smem - 1024 - (128 - p.xrows) * 128;
    p.D = p.pair ? 1 : p.n <= 64 && room / (4 * block) >= 4 ? 4 : p.n <= 128 && room / (2 * block) >= 4 ? 2 : 1;
    p.mc = (p.n / 16 + 2) / 3;
    if (p.D == 1 && p.mc < 3) p.mc = 3;  // (n is 96 or more)
    p.nbuf = 512 / (p.D * p.n) < 8 / p.D ? 512 / (p.D * p.n) : 8 / p.D;
    p.nst = room / (p.D * block);
    if (p.nst > kF8MaxStages) p.nst = kF8MaxStages;
    const int64_t tiles = (int64_t)p.RT * p.CT;
    p.grid = of * (int)(tiles < slots ? tiles : slots);
    return p;
}

int launch_fp8_gemm(const Fp8GemmCall& c, cudaStream_t st, cudaError_t* err);
int fp8_device_error(int clear);

}  // namespace mr
