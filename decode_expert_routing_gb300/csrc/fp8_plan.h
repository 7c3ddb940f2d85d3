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

// Tiles: rows of x are the accumulator's lanes (128 a CTA, of up to 64 rows 64;
// 256 a pair), n rows of w its columns.  slices > 1: CTAs of a cluster share
// a tile's blocks of K, slice_len each; every cluster has one tile.
struct Fp8Plan {
    int pair, n, xrows, RT, CT, D, mc, nst, nbuf, grid;  // mc: chunks of 16 columns of a read-back warp
    int slices, slice_len;
};
inline int fp8_room(int xrows) { return kF8Smem - 1024 - (128 - xrows) * 128; }  // for stages
// Blocks of a stage: as many as leave two buffers of accumulators and four stages.
inline int fp8_depth(bool pair, int xrows, int n) {
    const int block = (xrows + n) * 128, room = fp8_room(xrows);
    return pair ? 1 : n <= 64 && room / (4 * block) >= 4 ? 4 : n <= 128 && room / (2 * block) >= 4 ? 2 : 1;
}
inline int fp8_chunks(int n, int D) {  // of 16 columns, of a read-back warp (two groups)
    const int mc = (n / 16 + 1) / 2;
    return D > 1 ? mc : mc <= 4 ? 4 : mc <= 6 ? 6 : 7;
}
// Cycles of a block of K in one CTA, fitted to the times of every tile and
// number of slices at 21 sizes (off by 8 %, the chosen tile by 1 %, at most 4): the
// read-back, by its chunks and by how many blocks share its waits (four blocks of
// 48 columns 305, two of 96 460, one of 128 576, of 192 804; pairs of 192 655, of
// 224 716), or the bytes' way from L2, 57 a cycle (128 rows and 48 columns: 396).
inline int fp8_block_cycles(bool pair, int xrows, int n) {
    if (pair) return 290 + n * 19 / 10;
    const int D = fp8_depth(false, xrows, n), mc = fp8_chunks(n, D), l2 = (xrows + n) * 9 / 4;
    const int read = D == 4 ? 155 + 75 * mc : D == 2 ? 295 + 55 * mc : 120 + 114 * mc;
    return read > l2 ? read : l2;
}
// What a call costs besides: a pair's start and end, and handing the slices' sums over.
inline int fp8_call_cycles(bool pair, int n, int slices) {
    return pair ? 4900 : slices > 1 ? 38 * n + 570 * slices : 0;
}
// The tile and slices whose rounds cost least.  40 x 1536 x 6144: 48 columns in
// four slices 6.8 us, 32 in two 6.9, 16 in one 7.9; 40 x 6144 x 6144: 48 in one
// 10.0, 96 in two 11.5; 128 x 6144 x 6144: 96 in two 12.5, 64 in one 12.8; 700 x
// 1536 x 6144: 128 in two 12.6, 96 in one 16.4; 2048 x 1536 x 6144: 192 by pairs
// 20.6, by single CTAs 22.1; 4096 x 6144 x 6144 by pairs: 224 112, 192 120.
inline Fp8Plan fp8_plan(int M, int R, int K, int sms) {
    Fp8Plan p{};
    const int KI = (K + 127) / 128;
    int64_t least = INT64_MAX;
    for (int pair = 0; pair <= (M > 128 && sms >= 2 ? 1 : 0); ++pair) {
        const int of = 1 + pair, slots = sms / of, rt = (M + 128 * of - 1) / (128 * of);
        const int xrows = M >= 128 ? 128 : (M + 7) / 8 * 8;
        // (narrower pairs: twice as many single CTAs are faster)
        for (int n = 224; n >= (pair ? 160 : 16); n -= 16 * of) {
            const int ct = (R + n - 1) / n;
            const int64_t tiles = (int64_t)rt * ct;
            for (int s = 1; s <= (pair ? 1 : 8); s *= 2) {
                // (a slice is whole stages of up to four blocks, and every slice has one)
                const int len = s == 1 ? KI : ((KI + s - 1) / s + 3) / 4 * 4;
                if (s > 1 && (tiles * s > sms || len * (s - 1) >= KI)) break;
                const int64_t rounds = (tiles * s + slots - 1) / slots;
                const int64_t cost =
                    rounds * len * fp8_block_cycles(pair != 0, xrows, n) + fp8_call_cycles(pair != 0, n, s);
                if (cost >= least) continue;
                least = cost;
                p.pair = pair, p.n = n, p.xrows = xrows, p.RT = rt, p.CT = ct, p.slices = s, p.slice_len = len;
            }
        }
    }
    const int of = 1 + p.pair, block = (p.xrows + p.n / of) * 128, slots = sms / of;
    p.D = fp8_depth(p.pair != 0, p.xrows, p.n);
    p.mc = fp8_chunks(p.n, p.D);
    p.nbuf = 512 / (p.D * p.n) < 8 / p.D ? 512 / (p.D * p.n) : 8 / p.D;
    p.nst = fp8_room(p.xrows) / (p.D * block);
    if (p.nst > kF8MaxStages) p.nst = kF8MaxStages;
    const int64_t tiles = (int64_t)p.RT * p.CT;
    p.grid = p.slices > 1 ? (int)tiles * p.slices : of * (int)(tiles < slots ? tiles : slots);
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
