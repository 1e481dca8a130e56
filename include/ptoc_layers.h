/*
 * ptoc_layers.h - layer operators of libptoc.so that stand next to the window
 * collectives of ptoc.h: the norms around a block whose output is spread over
 * N windows, 8-bit activation checkpoints, and a mixture-of-experts layer for
 * a few tokens.
 *
 * The conventions of ptoc.h hold: device pointers on the current device,
 * asynchronous work on `stream`, row pitches in elements, arguments checked on
 * the host before any CUDA call, a status returned and NOTHING launched on an
 * error, every buffer owned by the caller. A workspace is caller memory of at
 * least the stated bytes, aligned to 256 bytes, whose contents before and
 * after a call mean nothing; calls that can overlap need one each.
 * These calls take PTOC_F32, PTOC_F16 and PTOC_BF16 (PTOC_I32 is
 * PTOC_ERR_UNSUPPORTED). Sums, norm statistics and gradients of weights are
 * held in binary32; an element is rounded once, when it is stored.
 * Results do not depend on scheduling: the same call on the same GPU gives
 * the same bits. Rows are fastest where bases are 16-byte aligned (a
 * checkpoint's codes: 8-byte), pitches too and rows of whole 16-byte words; odd
 * pitches, lengths or weights cost up to half the speed, odd bases more (bases
 * and pitches of exponents, and gates of one number or one per row, cost
 * nothing). One operand decides for the call.
 */
#ifndef PTOC_LAYERS_H
#define PTOC_LAYERS_H

#include <stddef.h>
#include <stdint.h>

#include "ptoc.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Widest row the norms accept (elements). */
#define PTOC_NORM_MAX_COLS 32768
/* Columns that share one exponent in an 8-bit checkpoint. */
#define PTOC_CKPT_BLOCK 32
/* Limits of ptoc_moe_few_tokens. */
#define PTOC_MOE_MAX_TOKENS 64
#define PTOC_MOE_MAX_EXPERTS 1024
#define PTOC_MOE_MAX_TOP_K 16

/* A [rows, cols] matrix: element (i, j) at data[i * ld + j], ld >= cols. */
typedef struct {
    void* data;
    int64_t ld;
} ptoc_matrix;

/* A [rows, cols] matrix held in 8 bits. Columns [32 b, 32 b + 32) of a row
 * share the power of two 2^(exps[i * ld_exps + b] - 127), the smallest one
 * with |x| <= 127 * 2^e for every x of the block (byte 0 where that, or the
 * block itself, is smaller); codes[i * ld_codes + j] = x / 2^e rounded to the
 * nearest integer, ties to even. The division is exact, so the codes do not
 * depend on how it is computed, and a restored value (code * 2^e) has at most
 * 7 significant bits: it is exact in every element type where it is in that
 * type's range (a value within 2^-7 of the largest float can round up to 2^128
 * and come back as infinity). A block that holds an infinity or a NaN has
 * exponent byte 255 and is restored as NaN. ld_codes >= cols, ld_exps >= ceil(cols / 32). */
typedef struct {
    int8_t* codes;
    int64_t ld_codes;
    uint8_t* exps;
    int64_t ld_exps;
} ptoc_ckpt8;

/* ptoc_checkpoint8 - x [rows, cols] -> out. x and out must not overlap. Both
 * calls take up to 2^31 - 256 columns and 2^31 - 1 pieces of 256 columns (rows
 * * ceil(cols / 256)), else PTOC_ERR_UNSUPPORTED. */
ptoc_status ptoc_checkpoint8(const ptoc_matrix* x, const ptoc_ckpt8* out, int64_t rows, int64_t cols,
                             ptoc_dtype dtype, cudaStream_t stream);

/* ptoc_restore8 - in -> x [rows, cols]. x and in must not overlap. */
ptoc_status ptoc_restore8(const ptoc_ckpt8* in, const ptoc_matrix* x, int64_t rows, int64_t cols,
                          ptoc_dtype dtype, cudaStream_t stream);

/* What the forward and backward pass of ptoc_block_norm share. */
typedef struct {
    int32_t post_norm;           /* 1: norm after the block; 0: n = a */
    int32_t param_dtype;         /* element type of the weights and the gate: dtype or PTOC_F32 */
    const void* post_weight;     /* [cols], or null for ones */
    const void* pre_weight;      /* [cols], or null for ones */
    const void* gate;            /* null for 1; else g(i, j) = gate[i * gate_row_stride + j * gate_col_stride] */
    int64_t gate_row_stride;     /* 0: the same for every row */
    int64_t gate_col_stride;     /* 0: the same for every column; else 1 */
    float residual_scale;
    float branch_scale;
    float eps;                   /* > 0 */
} ptoc_block_norm_params;

/*
 * ptoc_block_norm - the end of one block and the start of the next, in one
 * pass over the rows. For every row, with sums over its `cols` columns:
 *   a = parts[0] + parts[1] + ...      in rank order, as PTOC_SUM of ptoc_treduce
 *   n = a * ra * post_weight           ra = 1 / sqrt(mean(a^2) + eps); without
 *                                      the norm after the block n = a, ra = 1
 *   s = residual_scale * x + branch_scale * g * n          the residual stream
 *   y = s * r * pre_weight             r = 1 / sqrt(mean(s^2) + eps)
 * parts->root is ignored; all parts have the pitch ld_parts.
 * Outputs: out (s) is required. normed (y), block_out (a), block_ckpt (a in 8
 * bits), stream_ckpt (s as stored in out, in 8 bits) and rstd ([2, rows]
 * floats: ra, then r) may be null. y is computed from s before its rounding.
 * out may be exactly the residual x (same pointer and pitch); other overlaps
 * of an output are PTOC_ERR_ALIAS. cols above PTOC_NORM_MAX_COLS is
 * PTOC_ERR_UNSUPPORTED. An empty matrix is PTOC_OK without a launch.
 */
ptoc_status ptoc_block_norm(const ptoc_group* parts, int64_t ld_parts, const ptoc_matrix* x,
                            const ptoc_block_norm_params* params, const ptoc_matrix* out,
                            const ptoc_matrix* normed, const ptoc_matrix* block_out,
                            const ptoc_ckpt8* block_ckpt, const ptoc_ckpt8* stream_ckpt, float* rstd,
                            int64_t rows, int64_t cols, ptoc_dtype dtype, cudaStream_t stream);

/* What the backward pass reads of the forward pass: a and s, each either as a
 * matrix of the element type or as an 8-bit checkpoint (of a matrix and its
 * checkpoint exactly one has a non-null address), and the statistics rstd
 * ([2, rows]). */
typedef struct {
    ptoc_matrix block, stream;
    ptoc_ckpt8 block_ckpt, stream_ckpt;
    const float* rstd;
} ptoc_block_norm_saved;

/*
 * ptoc_block_norm_backward - the gradients of ptoc_block_norm. With dy the
 * gradient of normed and du the gradient that reaches out from elsewhere
 * (null: none):
 *   ds = du + r * (pre_weight * dy) - s * r^3 / cols * sum(pre_weight * dy * s)
 *   d_residual = residual_scale * ds            dn = branch_scale * g * ds
 *   d_block = ra * (post_weight * dn) - a * ra^3 / cols * sum(post_weight * dn * a)
 *             (the gradient of every part); d_block = dn without the norm after
 *   d_pre_weight  = sum over rows of dy * s * r                 [cols] floats
 *   d_post_weight = sum over rows of dn * a * ra                [cols] floats
 *   d_gate = branch_scale * ds * n, summed over the axes along which the gate
 *            is broadcast: floats, [rows, cols], [rows], [cols] or [1], packed
 * d_pre_weight, d_post_weight and d_gate may be null. d_post_weight needs the
 * norm after the block and d_gate a gate (else PTOC_ERR_INVALID_ARG).
 * d_residual may be exactly du, and d_block exactly block (both by pointer and
 * pitch); other overlaps of an output are PTOC_ERR_ALIAS. Limits as
 * ptoc_block_norm. With rows == 0 or cols == 0 the gradients of the weights and
 * of the gate, sums over nothing, are set to zero.
 */
size_t ptoc_block_norm_backward_workspace(int64_t rows, int64_t cols);
ptoc_status ptoc_block_norm_backward(const ptoc_block_norm_saved* saved, const ptoc_block_norm_params* params,
                                     const ptoc_matrix* dy, const ptoc_matrix* du,
                                     const ptoc_matrix* d_residual, const ptoc_matrix* d_block,
                                     float* d_pre_weight, float* d_post_weight, float* d_gate,
                                     void* workspace, size_t workspace_bytes,
                                     int64_t rows, int64_t cols, ptoc_dtype dtype, cudaStream_t stream);

/* How router logits become scores. */
typedef enum {
    PTOC_SCORE_SOFTMAX = 0,      /* over all experts */
    PTOC_SCORE_SIGMOID = 1
} ptoc_moe_score;

/* The layer's weights, packed, in the call's dtype unless said otherwise. One
 * rank of an expert-parallel group holds experts [first_expert, first_expert +
 * local_experts) of `experts`. */
typedef struct {
    const void* router;          /* [experts, hidden] of router_dtype */
    const float* bias;           /* [experts], added to the score for the choice only; or null */
    const void* w_in;            /* [local_experts, 2 * inter, hidden]: gate rows, then up rows */
    const void* w_out;           /* [local_experts, hidden, inter] */
    int32_t router_dtype;        /* dtype or PTOC_F32 */
    int32_t experts, first_expert, local_experts;
    int32_t top_k;
    int32_t score;               /* ptoc_moe_score */
    int32_t renormalize;         /* 1: the chosen weights sum to 1 (before scale) */
    float scale;
} ptoc_moe_params;

/*
 * ptoc_moe_few_tokens - a mixture-of-experts layer for 0 to 64 tokens: router,
 * choice, gated experts and weighted sum. For every token row x:
 *   logits = router x                                       binary32
 *   key    = logits (softmax without bias), else score + bias
 *   ids    = the top_k experts by descending key, ties to the lowest index; a
 *            NaN key counts as the lowest
 *   w      = score(ids), divided by their sum if renormalize, times scale
 *   y      = sum over the chosen local experts e of
 *            w_e * w_out[e] (silu(w_gate[e] x) * (w_up[e] x))
 * Rows none of whose experts are local are zero: the ranks' y are the parts
 * that ptoc_block_norm (or ptoc_allreduce) sums. The hidden activations
 * w_e * silu(..) * (..) enter the second product as two numbers of dtype whose
 * sum keeps 16 (bf16) or 22 (f16) significant bits, in f16 down to steps of
 * 2^-35; y is rounded once.
 * ids ([tokens, top_k] int32) and weights ([tokens, top_k] floats) may be null.
 * dtype is PTOC_F16 or PTOC_BF16 (PTOC_F32 is PTOC_ERR_UNSUPPORTED).
 * An f16 hidden activation beyond 65504 becomes infinite. An infinity or a NaN in x
 * stays with its token, and one in an expert's weights with the tokens that
 * chose the expert.
 * y must not overlap an input. tokens, experts or top_k above the limits are
 * PTOC_ERR_UNSUPPORTED. 16-byte aligned x, router and weights with hidden and
 * inter multiples of 8 take the tensor-core kernel: one cooperative launch,
 * whose waits for copies are bounded by PTOC_WAIT_NS (ptoc.h) and counted by
 * ptoc_wait_faults if they give up (part of y is then missing). Others take
 * plain kernels.
 */
size_t ptoc_moe_few_tokens_workspace(int64_t tokens, int64_t hidden, int64_t inter, int32_t experts, int32_t top_k);
ptoc_status ptoc_moe_few_tokens(const ptoc_matrix* x, const ptoc_moe_params* params, const ptoc_matrix* y,
                                int32_t* ids, float* weights, void* workspace, size_t workspace_bytes,
                                int64_t tokens, int64_t hidden, int64_t inter, ptoc_dtype dtype,
                                cudaStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* PTOC_LAYERS_H */
