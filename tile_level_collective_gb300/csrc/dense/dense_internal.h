// Parameter blocks and launchers of the dense block's operators (see
// ptoc_dense.h).
#pragma once

#include <cstddef>
#include <cstdint>

#include "layers/layers_internal.h"
#include "ptoc_dense.h"
#include "ptoc_internal.h"

namespace ptoc {

// ---- layer norm -----------------------------------------------------------------

struct LayerNormParams {
    const void* part[kMaxRanks];
    int64_t ld_part;
    const void* x;                       // may be null
    int64_t ld_x;
    void *out, *normed;                  // out may be null
    int64_t ld_out, ld_normed;
    const void *weight, *bias;           // may be null
    float* stats;                        // may be null
    int64_t rows, cols;
    int64_t step_part, step_x;           // elements from a block's row to its next one
    float eps, inv_cols;
    int32_t nparts, param_f32, access;   // Access
};

struct LayerNormBackParams {
    const void *s, *dy, *du;             // du may be null
    int64_t ld_s, ld_dy, ld_du;
    void* dx;
    int64_t ld_dx;
    const void* weight;                  // may be null
    const float* stats;
    float *d_weight, *d_bias;            // may be null
    float* partial;                      // the blocks' column sums: [2][grid, cols]
    int64_t rows, cols;
    int64_t step_s, step_dy, step_du;    // elements from a block's row to its next one
    float inv_cols;
    int32_t param_f32, access, grid;
};

// Blocks of the backward pass: each leaves two partial rows of column sums.
int layer_norm_backward_grid(int64_t rows, int64_t cols);

cudaError_t launch_layer_norm(const LayerNormParams& p, int dtype, cudaStream_t s);
cudaError_t launch_layer_norm_backward(const LayerNormBackParams& p, int dtype, cudaStream_t s);

// ---- the gated feed-forward block --------------------------------------------------

struct FfnParams {
    const void *x, *w_in, *w_out;
    int64_t ld_x, ld_in, ld_out;
    void *y, *pre;                       // pre may be null
    int64_t ld_y, ld_pre;
    char* ws;
    int64_t tokens, hidden, inter;
    int32_t act, vec;                    // vec: every matrix can be addressed in 16-byte words
    int32_t parts;                       // 2: two numbers for h at any number of tokens
};

struct FfnBackParams {
    const void *x, *pre, *w_in, *w_out, *dy;
    int64_t ld_x, ld_pre, ld_in, ld_out, ld_dy;
    void *dx, *d_in, *d_out;             // may be null
    int64_t ld_dx, ld_din, ld_dout;
    char* ws;
    int64_t tokens, hidden, inter;
    int32_t act, vec;
    int32_t parts;                       // 2: two numbers for dg, du and h in every product
};

// Rows of the workspace's activations begin at multiples of 16 bytes.
inline int64_t padded_inter(int64_t inter) { return (inter + 7) / 8 * 8; }

size_t ffn_workspace_bytes(int64_t tokens, int64_t hidden, int64_t inter);
size_t ffn_backward_workspace_bytes(int64_t tokens, int64_t hidden, int64_t inter);
cudaError_t launch_ffn(const FfnParams& p, int dtype, cudaStream_t s);
cudaError_t launch_ffn_backward(const FfnBackParams& p, int dtype, cudaStream_t s);
// The waits of the tensor-core kernels that gave up since the last call.
cudaError_t take_stage_faults_ffn_f16(uint32_t* count);
cudaError_t take_stage_faults_ffn_bf16(uint32_t* count);

// ---- the gradients' norm -------------------------------------------------------------

size_t clip_workspace_bytes(int32_t count);
cudaError_t launch_clip(const ptoc_gradient* grads, int32_t count, float max_norm, float* result, double* partial,
                        cudaStream_t s);

}  // namespace ptoc
