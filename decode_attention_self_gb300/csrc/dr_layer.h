// Internal declarations of the operators between a layer's attention calls (matrix product with an epilogue, residual
// norm).  Launch helpers take validated arguments; dr_layer_api.cu owns all argument checking.
#pragma once

#include <cuda.h>

#include "dr_prompt.h"   // once_per_device

namespace dr {

struct LinearOut {
    void *ptr;
    int64_t stride;   // elements between tokens
    int32_t col0;     // its first column
    int32_t cols;
};

struct LinearParams {
    const uint16_t *x;        // [T][K] bf16, tokens x_stride elements apart
    int64_t x_stride;
    const uint16_t *W;        // [N][K] bf16, or [2N][K] (gated: rows N.. are multiplied in)
    const uint16_t *bias;     // [N] or [2N] bf16, or null
    const void *residual;     // [T][N] of the outputs' type, tokens res_stride elements apart, or null
    int64_t res_stride;
    LinearOut out[DR_LINEAR_MAX_OUTS];
    int32_t n_outs;
    int32_t T, K, N;          // N: output columns
    int32_t act, gated;
    int32_t out_f32;
    int32_t vec_out, vec_res; // 1: rows of all outputs (there is a residual, and its rows) start on 16 bytes
    int32_t *err;
    int32_t stall_tile = -1;  // test hook: the CTAs of this output tile never load their first K chunk
};

// Tensor map of a bf16 or fp32 matrix [rows][cols], rows `stride` elements apart: boxes of box_rows x box_cols (128 or 64
// bytes, and the swizzle of that width), zeros outside.
bool encode_matrix(CUtensorMap *map, const void *ptr, bool f32, int64_t rows, int cols, int64_t stride, int box_rows,
                   int box_cols);

// Output tiles of a launch as the test hook counts them; 0 where the call runs a kernel without waits.
int linear_tiles(const LinearParams &p, int sms);
cudaError_t launch_linear(const LinearParams &p, cudaStream_t stream);
// Up to 32 tokens.
cudaError_t launch_linear_rows(const LinearParams &p, int sms, cudaStream_t stream);
cudaError_t launch_linear_cluster(const LinearParams &p, int sms, cudaStream_t stream);
int linear_cluster_tiles(const LinearParams &p, int sms);
bool linear_cluster_takes(const LinearParams &p, int sms);   // whether its tiles and accumulators suffice
cudaError_t launch_linear_tiles(const LinearParams &p, int sms, cudaStream_t stream);
int linear_tiles_tiles(const LinearParams &p, int sms);

struct NormParams {
    int32_t kind;             // DR_NORM_*
    float eps;
    const uint16_t *weight;   // [Dm] bf16 or null (ones)
    const uint16_t *bias;     // [Dm] bf16 or null (zeros)
};

struct ResidualNormParams {
    const void *x;            // [T][Dm]
    const void *residual;     // or null
    void *h;                  // or null
    void *y;                  // or null
    const uint16_t *gate;     // [Dm] (gate_stride 0) or [T][Dm], or null
    int64_t x_stride, res_stride, h_stride, y_stride, gate_stride;
    int32_t x_f32, res_f32, y_f32;
    float scale;
    NormParams post, pre;
    int32_t T, Dm;
};

cudaError_t launch_residual_norm(const ResidualNormParams &p, cudaStream_t stream);

}  // namespace dr
