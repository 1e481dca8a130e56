// Parameter blocks and launchers of the layer operators (see ptoc_layers.h).
#pragma once

#include <cstddef>
#include <cstdint>

#include "ptoc_internal.h"
#include "ptoc_layers.h"

namespace ptoc {

struct Ckpt;

// How rows can be read: at any address, at any pitch from 16-byte aligned
// bases, or in 16-byte aligned words throughout.
enum Access : int { kAnywhere = 0, kOddPitch = 1, kAligned = 2 };

struct Ckpt8Params {
    void* x;
    int64_t ld;
    ptoc_ckpt8 ckpt;
    int64_t rows, cols;
    int32_t access;               // Access; kOddPitch: the codes' rows are 8-byte aligned, x anywhere
};

// The element types of the norms' parameters are dtype, or binary32 where
// param_f32 is set.
struct NormCommon {
    const void *post_weight, *pre_weight, *gate;
    int64_t gate_rs, gate_cs;
    int32_t post_norm, param_f32;
    float residual_scale, branch_scale, eps, inv_cols;
    int64_t rows, cols;
    int32_t access;               // Access
};

struct NormParams {
    const void* part[kMaxRanks];
    NormCommon c;
    int64_t ld_part;
    const void* x;
    int64_t ld_x;
    void *out, *normed, *block_out;      // normed and block_out may be null
    int64_t ld_out, ld_normed, ld_block;
    ptoc_ckpt8 block_ckpt, stream_ckpt;  // codes null: not written
    float* rstd;                         // may be null
    int64_t step_part, step_x;           // elements from a block's row to its next one
    int32_t nparts;
};

struct NormBackParams {
    NormCommon c;
    const void *block, *stream;          // null: read from the checkpoint
    int64_t ld_block, ld_stream;
    ptoc_ckpt8 block_ckpt, stream_ckpt;
    const float* rstd;
    const void *dy, *du;                 // du may be null
    int64_t ld_dy, ld_du;
    void *d_residual, *d_block;
    int64_t ld_dres, ld_dblk;
    float *d_pre, *d_post, *d_gate;      // may be null
    float* partial;                      // the blocks' column sums: [2][grid, cols], then [grid] scalars
    int32_t gate_kind;                   // GateKind of d_gate
    int32_t need_q;                      // the second column sum is asked for
    int64_t step_stream, step_block, step_dy, step_du;       // bytes from a block's row to its next one
    int32_t grid;
};

enum GateKind : int { kGateNone = 0, kGateScalar = 1, kGateChannel = 2, kGateToken = 3, kGateElement = 4 };

// Blocks of the backward pass: each leaves two partial rows of column sums
// and a scalar in the workspace.
int norm_backward_grid(int64_t rows, int64_t cols);

cudaError_t launch_checkpoint8(const Ckpt8Params& p, int dtype, cudaStream_t s);
cudaError_t launch_restore8(const Ckpt8Params& p, int dtype, cudaStream_t s);
cudaError_t launch_block_norm(const NormParams& p, int dtype, cudaStream_t s);
cudaError_t launch_block_norm_backward(const NormBackParams& p, int dtype, cudaStream_t s);

struct MoeParams {
    const void *x, *router, *w_in, *w_out;
    const float* bias;
    void* y;
    int64_t ld_x, ld_y;
    int32_t* ids;                        // user outputs, may be null
    float* weights;
    char* ws;                            // workspace
    int64_t hidden, inter;
    int32_t tokens, experts, first, local, top_k;
    int32_t router_f32, sigmoid, renormalize, vec;
    float scale;
};

size_t moe_workspace_bytes(int64_t tokens, int64_t hidden, int64_t inter, int experts, int top_k);
cudaError_t launch_moe_few(const MoeParams& p, int dtype, cudaStream_t s);
// The waits of the mixture-of-experts kernel that gave up since the last call.
cudaError_t take_stage_faults_moe(uint32_t* count);

}  // namespace ptoc
