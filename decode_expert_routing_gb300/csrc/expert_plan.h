// Host-side shape of the expert products and the launcher's arguments.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace mr {

// Tiles of a weight [R, K]: RT tiles of 128 rows (gate/up: of 64 features,
// both of their rows), KI k-blocks of 128 code bytes a row, W scale words per
// row and k-block.
struct ExpertShape {
    int RT, KI, W;
};
inline ExpertShape expert_shape(int R, int K, bool fp4, bool gate_up) {
    ExpertShape s;
    s.RT = gate_up ? (R / 2 + 63) / 64 : (R + 127) / 128;
    s.KI = fp4 ? (K + 255) / 256 : (K + 127) / 128;
    s.W = fp4 ? 2 : 1;
    return s;
}

// Scratch of a down call: its products of mk assignments, rows of R, rounded to
// bf16 (half a step, 2^-8 of each), or the upper halves of the fp32 products,
// whose lower halves have a buffer as large.  Written and read once, they are
// the call's largest traffic next to the weights.  128 experts x 6144 x 768,
// E4M3, top-8, rounded and whole: 1 token 12.6 and 12.9 us, 64 tokens 82.1 and
// 83.7, 256 101 and 105, 1001 127 and 164, 4096 260 and 417.
inline size_t expert_scratch_bytes(int64_t mk, int R) { return ((size_t)mk * (size_t)R * 2 + 255) / 256 * 256; }

// Whether two CTAs share their activation rows (256 weight rows a tile): where
// an expert has 16 rows or more on average, and there are 64 in all.  Gate/up
// of 1001 tokens x 8 over 128 experts, E2M1: 119 us as pairs, 139 alone; of 256
// tokens, E4M3: 190 and 199; of 128: 177 and 176.  A product of 64 rows with
// 6144 x 6144, E4M3, not split: 12.2 and 12.7; of 33, E2M1: 7.8 and 7.6.
inline bool expert_pair(int64_t mk, int E) { return mk >= 64 && mk >= 16 * (int64_t)E; }

// CTAs that share a tile's K range (1: none do), where the tiles leave SMs
// without work: 2, 4 or 8 (clusters of 3 and 6 were placed so that some had to
// wait), with a tile for every cluster; *len is each one's k-blocks, a multiple
// of those whose scales are 16 bytes of a row.  A k-block takes 0.2 us or more;
// handing the sums over 1.5 us and the columns' way through distributed shared
// memory (some 90 bytes a cycle for a cluster).  64 x 500 x 6144, E4M3: 6.7 us
// in slices, 11.2 in one; 33 x 6144 x 6144: 10.4 in 2, 12.2 in one.
inline int expert_slices(int64_t mk, int E, const ExpertShape& s, int ctas, int* len) {
    // (a run of blocks has at most 15 rows more than assignments)
    const int64_t hit = mk < E ? mk : E, tiles = (hit + (mk + 15 * hit) / 256) * s.RT;
    const int64_t rows = mk / hit < 256 ? mk / hit : 256;
    const int group = 4 / s.W;
    int best = 1;
    double most = 0.0;
    *len = s.KI;
    for (int n = 2; n <= 8; n *= 2) {
        if (tiles * n * 10 > (int64_t)ctas * 9) break;
        const int l = ((s.KI + n - 1) / n + group - 1) / group * group;
        const double gain = 0.2 * (s.KI - l) - 1.5 - 0.003 * (double)rows * (n - 1);
        if ((int64_t)l * (n - 1) < s.KI && gain > most) most = gain, best = n, *len = l;  // (every slice has k-blocks)
    }
    return best;
}

// Rows of a gemm's column tiles (a multiple of 16, of 32 for pairs; at most
// 256): of the sizes, the one whose rounds of tiles cost least, a round taken
// as 256 + rows (the loads of a stage: its weight rows and its activation
// rows).  4096 x 6144 x 6144, E2M1: tiles of 224 rows, 6 full rounds, 50.4 us;
// of 256, 5.05 of 6 rounds, 52.9.
// Where slices CTAs share a tile, the clusters are all there is: one round, which
// tiles of 256 rows fit (expert_slices) and is cheaper than any two.
inline int expert_gemm_rows(int M, int RT, bool pair, int slices, int ctas) {
    const int step = pair ? 32 : 16;
    if (M <= 256) return (M + step - 1) / step * step;
    const int slots = ctas / (pair ? 2 : slices), rows = pair ? (RT + 1) / 2 : RT;
    int best = 256;
    int64_t least = INT64_MAX;
    for (int per = 256; per >= 128; per -= step) {
        const int64_t tiles = ((int64_t)M + per - 1) / per * rows, cost = (tiles + slots - 1) / slots * (256 + per);
        if (cost < least) least = cost, best = per;
    }
    return best;
}

// One launch of the expert kernel (op: 0 gemm, 1 gate/up, 2 down).
struct ExpertCall {
    int op, fp4, gather, out_fmt;  // out_fmt: 0 bf16, 1 MXFP8, 2 MXFP4, 3 fp32
    int E, R, K, M, topk, nblk, block;
    const uint8_t *w, *w_scale, *x, *x_scale;
    int64_t ldx, lds, ldo, x_rows;
    const int32_t *sorted, *experts, *topk_ids;
    const float* topk_weights;
    const void* add;
    void* out;
    uint8_t* out_scale;
    void *scratch, *scratch_low;
};
int launch_expert(const ExpertCall& c, cudaStream_t st, cudaError_t* err);
cudaError_t launch_mx_pack(const uint8_t* scale, int64_t E, int R, int K, int fp4, int gate_up, void* packed,
                           cudaStream_t st);
int expert_device_error(int clear);

}  // namespace mr
