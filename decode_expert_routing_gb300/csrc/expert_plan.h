// Host-side shape of the expert products and the launcher's arguments.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace mr {

// Tiles of a weight [R, K]: RT tiles of 128 rows (gate/up: of 64 features,
// both of their rows), KI stages of 128 code bytes, W scale words per row and
// stage.
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

// Scratch of a down call: its products of mk assignments in bf16, rows of R.
inline size_t expert_scratch_bytes(int64_t mk, int R) { return ((size_t)mk * (size_t)R * 2 + 255) / 256 * 256; }

// Whether two CTAs share their activation rows (256 weight rows a tile): where
// an expert has 16 rows or more on average (256 tokens x 8 over 128 experts,
// E4M3 gate/up: 199 us as pairs, 252 alone) and there is a tile for every CTA.
inline bool expert_pair(int64_t mk, int E, int RT, int ctas) {
    const int64_t tiles = ((mk < E ? mk : E) + mk / 256) * RT;
    return mk >= 16 * (int64_t)E && tiles >= ctas;
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
    void* scratch;
};
int launch_expert(const ExpertCall& c, cudaStream_t st, cudaError_t* err);
cudaError_t launch_mx_pack(const uint8_t* scale, int64_t E, int R, int K, int fp4, int gate_up, void* packed,
                           cudaStream_t st);
int expert_device_error(int clear);

}  // namespace mr
