// Host-side plan of the FP8 product with scales per 128.
#pragma once

#include <cuda.h>
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

// Few rows of x: CTAs of 16 A rows of w and 8 B rows of x, gx x gy of them, nst
// stages a warp.
constexpr int kF8FewStages = 8;
constexpr int kF8FewSmem = 220 * 1024;
struct Fp8FewPlan {
    int A, B, gx, gy, nst, smem;
};
inline bool fp8_few(int M) { return M <= 16; }
inline Fp8FewPlan fp8_few_plan(int M, int R, int K, int sms) {
    Fp8FewPlan p{};
    p.B = M <= 8 ? 1 : 2;
    p.A = (R + 31) / 32 >= sms ? 2 : 1;
    p.gx = (R + 16 * p.A - 1) / (16 * p.A);
    p.gy = (M + 8 * p.B - 1) / (8 * p.B);
    const int KI = (K + 127) / 128, stage = (16 * p.A + 8 * p.B) * 128, per = (KI + 7) / 8;
    // two CTAs on an SM where there are more than SMs
    p.nst = ((int64_t)p.gx * p.gy > sms ? 110 * 1024 : kF8FewSmem - 1024) / (8 * stage);
    if (p.nst > kF8FewStages) p.nst = kF8FewStages;
    if (p.nst > per) p.nst = per;
    const int ring = 8 * p.nst * stage, sums = 8 * 8 * p.B * (16 * p.A + 1) * 4;
    p.smem = (ring > sums ? ring : sums) + 1024;
    return p;
}
int launch_fp8_few(const Fp8GemmCall& c, int sms, cudaStream_t st, cudaError_t* err);
int fp8_few_device_error(int clear);

// Rows of K bytes, boxes of box_rows x 128 bytes in the 128-byte swizzle; behind K and the last row zeros are read.
bool fp8_encode(CUtensorMap* map, const void* ptr, int K, int64_t rows, int64_t ld, int box_rows);

int launch_fp8_gemm(const Fp8GemmCall& c, cudaStream_t st, cudaError_t* err);
int fp8_device_error(int clear);

}  // namespace mr
