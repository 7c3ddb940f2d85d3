// Host-side arguments and launchers of the rows that move between the tokens
// and the sort's positions.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace mr {

enum { kRowBf16 = 0, kRowFp16 = 1, kRowFp32 = 2, kRowU8 = 3 };
inline int row_elem_bytes(int type) { return type == kRowFp32 ? 4 : type == kRowU8 ? 1 : 2; }

// To the experts: out[p] = weights[f] x[f / topk] (weights null: the row as it
// is), f = sorted[p]; with y, grad_w[f] = <x[f / topk], y[p]>.
struct ToExpertsArgs {
    const void *x, *y;
    int64_t ldx, ldy;      // elements
    const float* weights;  // [mk]
    const int32_t *sorted, *npost;
    const int32_t* ids;    // with positions: [mk]
    int32_t* positions;    // [mk], or null
    const int32_t* known;  // with grad_w: positions [mk]
    float* grad_w;         // [mk], or null
    void* out;             // [cap, K]
    int64_t cap;
    int M, K, topk, E, type;
    int row_bytes;         // of a row; this, x_bytes and y_bytes, from the first row's start to the last one's
    int64_t x_bytes, y_bytes;  // end, are set by the launcher
};
// Back to the tokens: out[m] = add[m] + sum_j weights[m, j] y[positions[m, j]].
struct ToTokensArgs {
    const void *y, *add;
    int64_t ldy, ldadd, cap;
    const int32_t* positions;
    const float* weights;  // or null: ones
    void* out;             // [M, K]
    int M, K, topk, type;
    int row_bytes;         // of a row; this, y_bytes and add_bytes, from the first row's start to the last one's
    int64_t y_bytes, add_bytes;  // end, are set by the launcher
};
cudaError_t launch_to_experts(const ToExpertsArgs& a, cudaStream_t st);
cudaError_t launch_to_tokens(const ToTokensArgs& a, cudaStream_t st);

}  // namespace mr
