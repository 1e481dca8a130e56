/*
 * ptoc_dense.h - operators of libptoc.so for the training and serving step of
 * a dense block whose output is spread over N windows: layer norm of the
 * windows' sum, the gated feed-forward block, each with its backward pass, and
 * the global norm of the gradients with clipping.
 *
 * The conventions of ptoc_layers.h hold: device pointers on the current
 * device, asynchronous work on `stream`, row pitches in elements, arguments
 * checked on the host before any CUDA call, a status returned and NOTHING
 * launched on an error, every buffer owned by the caller. A workspace is caller
 * memory of at least the stated bytes, aligned to 256 bytes, whose contents
 * before and after a call mean nothing; calls that can overlap (two streams,
 * two captured graphs) need one each. Results do not depend on scheduling: the
 * same call on the same GPU gives the same bits.
 *
 * A call may be several launches. Until it has returned, no other thread may put
 * work on its stream that writes its operands or uses its workspace: such work
 * could come between two of them. (It would also be too late to be waited for: up
 * to 128 tokens the second launch of ptoc_gated_ffn and of its backward pass reads
 * weights before the launch in front of it in the stream has ended.) Work that the
 * thread put there before the call is waited for, whatever it writes.
 */
#ifndef PTOC_DENSE_H
#define PTOC_DENSE_H

#include <stddef.h>
#include <stdint.h>

#include "ptoc_layers.h"

#ifdef __cplusplus
extern "C" {
#endif

/* What the forward and backward pass of ptoc_layer_norm share. */
typedef struct {
    const void* weight;          /* [cols], or null for ones */
    const void* bias;            /* [cols], or null for zeros (not read by the backward pass) */
    int32_t param_dtype;         /* element type of both: dtype or PTOC_F32 */
    float eps;                   /* > 0 (not read by the backward pass) */
} ptoc_layer_norm_params;

/*
 * ptoc_layer_norm - the sum of a block's windows, its residual and its layer
 * norm in one pass over the rows. For every row, with sums over its columns:
 *   s    = x + (parts[0] + parts[1] + ...)     the parts in rank order; x null: without it
 *   mean = sum(s) / cols
 *   rstd = 1 / sqrt(sum((s - mean)^2) / cols + eps)
 *   y    = (s - mean) * rstd * weight + bias
 * parts->root is ignored; all parts have the pitch ld_parts.
 * Outputs: normed (y) is required; out (s) and stats ([2, rows] floats: mean,
 * then rstd) may be null. Statistics are binary32 (deviations from the mean,
 * not differences of squares) and, like y, of s before its rounding. PTOC_F32,
 * PTOC_F16 and PTOC_BF16; each output is rounded once. A row that holds an
 * infinity or a NaN is NaN in y; a finite one whose squared deviations add to
 * more than binary32 holds (a spread of 1e17 at the least) has rstd 0, and y is
 * the bias (NaN where the sum of s leaves binary32 too). out may be exactly x
 * (same pointer and pitch); other overlaps of an output are PTOC_ERR_ALIAS. cols
 * above PTOC_NORM_MAX_COLS is PTOC_ERR_UNSUPPORTED. An empty matrix is PTOC_OK
 * without a launch.
 */
ptoc_status ptoc_layer_norm(const ptoc_group* parts, int64_t ld_parts, const ptoc_matrix* x,
                            const ptoc_layer_norm_params* params, const ptoc_matrix* out, const ptoc_matrix* normed,
                            float* stats, int64_t rows, int64_t cols, ptoc_dtype dtype, cudaStream_t stream);

/*
 * ptoc_layer_norm_backward - the gradients of ptoc_layer_norm from the stream
 * s (as stored) and its statistics. With n = (s - mean) * rstd, dy the gradient
 * of normed and du the gradient that reaches the stream from elsewhere (null:
 * none):
 *   t  = weight * dy
 *   dx = du + rstd * (t - sum(t) / cols - n * sum(t * n) / cols)
 *        (the gradient of x and of every part)
 *   d_weight = sum over rows of dy * n        [cols] floats
 *   d_bias   = sum over rows of dy            [cols] floats
 * d_weight and d_bias may be null. dx may be exactly du or exactly dy; other
 * overlaps of an output are PTOC_ERR_ALIAS. Limits as ptoc_layer_norm. With
 * rows == 0 the gradients of weight and bias are set to zero.
 */
size_t ptoc_layer_norm_backward_workspace(int64_t rows, int64_t cols);
ptoc_status ptoc_layer_norm_backward(const ptoc_matrix* s, const float* stats, const ptoc_layer_norm_params* params,
                                     const ptoc_matrix* dy, const ptoc_matrix* du, const ptoc_matrix* dx,
                                     float* d_weight, float* d_bias, void* workspace, size_t workspace_bytes,
                                     int64_t rows, int64_t cols, ptoc_dtype dtype, cudaStream_t stream);

/* The activation of a gated block, computed in binary32: act(g) is off by at most
 * 2^-19 of its value, act'(g) by as much of its two terms, for |g| up to 16 (silu
 * 2^-18 down to -80; what is below 2^-120 may be zero). */
typedef enum {
    PTOC_ACT_SILU = 0,           /* g / (1 + exp(-g)) */
    PTOC_ACT_GELU = 1            /* g * (1 + erf(g / sqrt(2))) / 2 */
} ptoc_act;

/* Limits of ptoc_gated_ffn and its backward pass. */
#define PTOC_FFN_MAX_TOKENS 4194304
#define PTOC_FFN_MAX_WIDTH 262144

/* The block's weights, in the call's dtype, and how many numbers of it what passes
 * between the products takes. One is what a tensor core reads: an output has the
 * error of two roundings (2.35e-3 of its norm in bf16, 2.9e-4 in f16). Two, the
 * second one what the first left, keep 16 (bf16) or 22 (f16, in steps of 2^-24 at the
 * least) significant bits: y and all gradients have the error of their own rounding
 * (1.65e-3, 2.1e-4), at any number of tokens, width and pitch, for 1.35 times the time
 * forward and 1.6 to 1.9 times backward (2.4 times below 128 tokens). A call with
 * parts = 2 needs twice the bytes of workspace that the functions below state. An
 * infinity in the weights, x or dy meets both numbers there, and may come out as NaN. */
typedef struct {
    ptoc_matrix w_in;            /* [2 * inter, hidden]: gate rows, then up rows */
    ptoc_matrix w_out;           /* [hidden, inter] */
    int32_t act;                 /* ptoc_act */
    int32_t parts;               /* 2; or 1 (or 0), where up to 64 tokens y and dx have 2 all the same */
} ptoc_gated_ffn_params;

/*
 * ptoc_gated_ffn - a gated feed-forward block. For every token row x [hidden]:
 *   [g, u] = w_in x
 *   h      = act(g) * u
 *   y      = w_out h
 * pre ([tokens, 2 * inter]: g, then u) is what the backward pass reads; null:
 * not kept. dtype is PTOC_F16 or PTOC_BF16 (others: PTOC_ERR_UNSUPPORTED). Sums
 * are binary32. Tensor cores cut them off where others round: in chains of at most
 * 32768 terms, whose sums are rounded, by 5e-5 of a long sum of random signs and
 * 2.5e-4 of one of one sign (in proportion less for shorter chains). h is taken from
 * g and u before their rounding and enters the second product rounded to dtype, as
 * a tensor core reads it; with two parts, and up to 64 tokens, as two numbers of
 * dtype whose sum keeps 16 (bf16) or 22 (f16) significant bits, or in binary32. y and
 * pre are rounded once. An infinity or a NaN in x stays with its token, and an f16 h
 * beyond 65504 becomes infinite unless it enters in binary32. Outputs must not
 * overlap anything (PTOC_ERR_ALIAS). Tokens above PTOC_FFN_MAX_TOKENS, hidden or
 * inter above PTOC_FFN_MAX_WIDTH are PTOC_ERR_UNSUPPORTED; tokens == 0 is PTOC_OK
 * without a launch.
 * 16-byte aligned matrices and pitches with hidden and inter multiples of 8 take
 * the tensor cores, in two launches; their waits for copies are bounded by
 * PTOC_WAIT_NS (ptoc.h) and counted by ptoc_wait_faults if they give up (part of
 * the outputs is then missing). Others take plain kernels, a hundred times slower
 * for long batches; two parts are binary32 there. A workspace serves all calls
 * of up to its tokens.
 */
size_t ptoc_gated_ffn_workspace(int64_t tokens, int64_t hidden, int64_t inter);
ptoc_status ptoc_gated_ffn(const ptoc_matrix* x, const ptoc_gated_ffn_params* params, const ptoc_matrix* y,
                           const ptoc_matrix* pre, void* workspace, size_t workspace_bytes, int64_t tokens,
                           int64_t hidden, int64_t inter, ptoc_dtype dtype, cudaStream_t stream);

/*
 * ptoc_gated_ffn_backward - the gradients of ptoc_gated_ffn, from x and pre. With
 * g and u as pre holds them and dy the gradient of y:
 *   dh    = dy w_out                       per token: w_out^T dy
 *   dg    = dh * u * act'(g)               du = dh * act(g)
 *   dx    = [dg, du] w_in
 *   d_w_in  = [dg, du]^T x                 [2 * inter, hidden]
 *   d_w_out = dy^T (act(g) * u)            [hidden, inter]
 * dx, d_w_in and d_w_out have the call's dtype; each may be null. dg, du and
 * act(g) * u enter the second products rounded to dtype (with two parts, and of up to
 * 64 tokens dg and du in dx's, as two numbers of it or in binary32); what is
 * beyond f16's range becomes infinite unless it enters in binary32. Outputs must not
 * overlap anything. Types, limits, waits and forms as ptoc_gated_ffn; up to three
 * launches (five of the plain kernels). With tokens == 0 the gradients of the
 * weights are set to zero.
 */
size_t ptoc_gated_ffn_backward_workspace(int64_t tokens, int64_t hidden, int64_t inter);
ptoc_status ptoc_gated_ffn_backward(const ptoc_matrix* x, const ptoc_matrix* pre, const ptoc_gated_ffn_params* params,
                                    const ptoc_matrix* dy, const ptoc_matrix* dx, const ptoc_matrix* d_w_in,
                                    const ptoc_matrix* d_w_out, void* workspace, size_t workspace_bytes,
                                    int64_t tokens, int64_t hidden, int64_t inter, ptoc_dtype dtype,
                                    cudaStream_t stream);

/* One gradient of a set: [rows, cols] elements at pitch ld, and where the
 * scaled ones go (null: in place). Elements between the rows stay as they are. */
typedef struct {
    void* data;
    void* out;
    int64_t ld, ld_out;
    int64_t rows, cols;
    int32_t dtype;               /* PTOC_F32, PTOC_F16 or PTOC_BF16, of data and out */
} ptoc_gradient;

/* Gradients of one call. */
#define PTOC_CLIP_MAX_GRADIENTS 65536

/*
 * ptoc_clip_gradients - the global norm of a set of gradients, and the set
 * scaled to at most max_norm:
 *   norm  = sqrt(sum of g^2 over every element of every gradient)
 *   scale = max_norm / (norm + 1e-6) if that is below 1, else 1
 *   g'    = scale * g, rounded once
 * result ([2] floats) receives norm and scale. Up to 32 squares are added in
 * binary32, scaled where that would overflow or underflow, and everything else
 * in binary64: the norm is finite whenever its value fits. With scale 1
 * gradients in place are not written, and those with an `out` are copied. A norm
 * that is infinite (one that binary32 cannot hold is) or NaN has scale 1: the
 * caller tells from result[0]. max_norm > 0; infinity asks for the norm alone.
 * Gradients and outs must not overlap one another, but for an out that is exactly
 * its own gradient (same pitch). More than PTOC_CLIP_MAX_GRADIENTS, or more than
 * 2^45 elements in all, are PTOC_ERR_UNSUPPORTED. count == 0 has norm 0.
 */
size_t ptoc_clip_gradients_workspace(int32_t count);
ptoc_status ptoc_clip_gradients(const ptoc_gradient* grads, int32_t count, float max_norm, float* result,
                                void* workspace, size_t workspace_bytes, cudaStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* PTOC_DENSE_H */
