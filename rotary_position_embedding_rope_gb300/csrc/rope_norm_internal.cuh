// rope_norm_internal.cuh -- declarations of the norm of query and key heads
// with the rotation in the same pass.  Not part of the public ABI.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "rope_serving.cuh"

namespace rope {

// CTAs of the backward kernel at most: a row of partial weight gradients each
// (nine for each of 152 SMs).
constexpr int32_t kNormPartials = 1368;

struct NormTensor {
    const void *x, *g, *w;           // rows, their output's gradient, weights [D] or nullptr
    void *y, *dw;                    // output, or gradient of the rows; gradient of the weights
    float *partial;                  // [CTAs][D], or nullptr: dw is not wanted
    int64_t xs[3], ys[3];            // strides of x, and of y and g: batch, token, head (elements)
    int32_t heads;
};

struct NormArgs {
    NormTensor t[2];                 // queries, keys (heads 0: none)
    const float *cos, *sin;
    const int32_t *pos;              // [S] or [B][pos_stride], or nullptr
    int64_t pos_stride;              // 0: one row for all sequences
    int64_t table_rows, tokens, B, S;
    int64_t tiles[2];
    int32_t D, rotary_dim, w_f32;
    float eps, inv_d;
    int32_t *flag;
};
cudaError_t launch_norm_f32(const NormArgs &a, int32_t layout, bool backward, cudaStream_t st);
cudaError_t launch_norm_bf16(const NormArgs &a, int32_t layout, bool backward, cudaStream_t st);
cudaError_t launch_norm_f16(const NormArgs &a, int32_t layout, bool backward, cudaStream_t st);

struct NormAppendArgs {
    RowsArgs rows;                   // keys, values, the pools, sequences and positions
    const void *q;                   // [total][Hq][D]
    int64_t q_stride;
    void *q_out;                     // [total][Hq][D], dense
    const void *wq, *wk;
    int32_t Hq, w_f32;
    float eps;
};
cudaError_t launch_norm_append_bf16(const NormAppendArgs &a, int32_t D, int32_t layout, cudaStream_t st);
cudaError_t launch_norm_append_f16(const NormAppendArgs &a, int32_t D, int32_t layout, cudaStream_t st);

}  // namespace rope
