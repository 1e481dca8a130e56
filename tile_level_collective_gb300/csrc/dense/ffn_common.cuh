// The forms of the gated feed-forward block.
#pragma once

#include <cstring>

#include "dense/dense_internal.h"

namespace ptoc {

// Up to this many tokens the products with weights take the form that streams them.
constexpr int64_t kFewTokens = 128;

// Stages (64 elements of depth) whose products are added by the tensor core alone. It
// cuts each sum off where the CUDA cores round it, so that a chain loses 1e-9 of its value
// for each element of depth (two parts 3e-9: the second one's small terms are cut off
// against the first one's sum). In one chain 262144 tokens lost 2.7e-4 of the weights'
// gradients, more than f16's rounding, and 4194304 tokens 4.3e-3.
constexpr int64_t kChain = 512;

// Up to this many tokens h, and dg and du on their way to dx, are kept in more bits
// than the type has: in two numbers of it, or in binary32.
constexpr int64_t kPartsTokens = 64;

// The forward pass' workspace holds h: of up to 64 tokens both parts, of 8, 16, 32
// or 64 rows each; of up to 128 tokens 128 rows. What serves more tokens serves
// fewer.
inline int64_t few_rows(int64_t tokens)
{
    int64_t rows = 8;
    while (rows < tokens) rows *= 2;
    return rows;
}
inline int64_t few_parts(int64_t tokens) { return tokens <= kPartsTokens ? 2 : 1; }

// The backward pass' workspace, in elements: dg's rows (all parts), du's `plane`
// elements after them, and h.
struct BackLayout {
    int64_t ld, plane, h, elements;
};
inline BackLayout back_layout(int64_t tokens, int64_t inter)
{
    BackLayout l;
    l.ld = padded_inter(inter);
    const int64_t rows = tokens <= kFewTokens ? few_rows(tokens) : tokens;
    l.plane = l.ld * rows * (tokens <= kFewTokens ? few_parts(tokens) : 1);
    l.h = 2 * l.plane;
    l.elements = l.h + l.ld * rows;
    return l;
}

// The same where every product takes two numbers for each (at most twice the bytes
// of the above): planes of dg, du and h, and planes of their second numbers.
inline BackLayout parts_layout(int64_t tokens, int64_t inter)
{
    BackLayout l;
    l.ld = padded_inter(inter);
    l.plane = l.ld * tokens;
    l.h = 2 * l.plane;
    l.elements = 6 * l.plane;
    return l;
}

// Any address and pitch.
cudaError_t launch_ffn_plain(const FfnParams& p, int dtype, cudaStream_t s);
cudaError_t launch_ffn_backward_plain(const FfnBackParams& p, int dtype, cudaStream_t s);

// 16-byte aligned rows of whole 16-byte words.
cudaError_t launch_ffn_tensor_f16(const FfnParams& p, cudaStream_t s);
cudaError_t launch_ffn_tensor_bf16(const FfnParams& p, cudaStream_t s);
cudaError_t launch_ffn_backward_tensor_f16(const FfnBackParams& p, cudaStream_t s);
cudaError_t launch_ffn_backward_tensor_bf16(const FfnBackParams& p, cudaStream_t s);

}  // namespace ptoc
