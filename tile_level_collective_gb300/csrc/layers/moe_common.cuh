// Pieces that both forms of the mixture-of-experts layer use.
#pragma once

#include "layers/layers_common.cuh"
#include "layers/layers_internal.h"

namespace ptoc {

__device__ __forceinline__ float warp_sum(float v)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// An activation on its way to the second product, as two numbers of the
// layer's type: high + low * kLowUnit. Their sum keeps 16 significant bits of
// bf16 and 22 of f16, so that the product's error is that of its result's
// rounding (with one number, an error of the same size came on top: 2.35e-3
// of the result's norm instead of 1.65e-3 in bf16). The unit keeps the lower
// part of small f16 activations (an expert's weight is a factor of them) above
// the smallest f16: steps of 2^-35 in place of 2^-24. One beyond the type's
// range, or a NaN, is the high part alone.
template <class T>
constexpr float kLowUnit = std::is_same<T, __half>::value ? 1.0f / 2048.0f : 1.0f;

template <class T>
struct Parts {
    T high, low;
    __device__ __forceinline__ float value() const { return fmaf(to_f32(low), kLowUnit<T>, to_f32(high)); }
};

template <class T>
__device__ __forceinline__ Parts<T> split_parts(float v)
{
    const T high = from_f32<T>(v);
    const float rest = (v - to_f32(high)) * (1.0f / kLowUnit<T>);       // exact; at most 2^15 in f16
    return Parts<T>{high, from_f32<T>(isfinite(rest) ? rest : 0.0f)};
}

// Floats in an order that unsigned comparison keeps, all above 1, which stands
// for NaN; 0 is left for "not there" and "taken".
__device__ __forceinline__ uint32_t ordered(float v)
{
    if (v != v) return 1u;
    if (v == 0.0f) v = 0.0f;               // -0 ties with +0
    const uint32_t u = __float_as_uint(v);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// One warp chooses for one token: top_k rounds of the largest key, lowest
// index first among equals. Lane l holds experts l, 32 + l, ... in registers
// (L of them). ids and weights are written by lane k for round k.
template <int L>
__device__ __forceinline__ void choose_experts(const MoeParams& m, const float* logits, int32_t* ids, float* weights)
{
    const int lane = threadIdx.x & 31, n = m.experts;
    float v[L];
    float top = -INFINITY, total = 0.0f;
#pragma unroll
    for (int j = 0; j < L; ++j) {
        const int e = j * 32 + lane;
        v[j] = e < n ? logits[e] : -INFINITY;
        top = fmaxf(top, v[j]);
    }
    if (!m.sigmoid) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
#pragma unroll
        for (int j = 0; j < L; ++j)
            if (j * 32 + lane < n) total += expf(v[j] - top);
        total = warp_sum(total);
    }
    auto score = [&](float x) { return m.sigmoid ? 1.0f / (1.0f + expf(-x)) : expf(x - top) / total; };
    uint32_t key[L];
#pragma unroll
    for (int j = 0; j < L; ++j) {
        const int e = j * 32 + lane;
        float k = v[j];
        if (e < n && (m.sigmoid || m.bias)) k = m.bias ? score(k) + m.bias[e] : score(k);
        key[j] = e < n ? ordered(k) : 0u;
    }
    int id = 0;
    for (int k = 0; k < m.top_k; ++k) {
        uint32_t best = 0;
        int at = INT32_MAX;
#pragma unroll
        for (int j = 0; j < L; ++j)
            if (key[j] > best) best = key[j], at = j * 32 + lane;
        const uint32_t high = __reduce_max_sync(0xffffffffu, best);
        at = __reduce_min_sync(0xffffffffu, best == high ? at : INT32_MAX);
#pragma unroll
        for (int j = 0; j < L; ++j)
            if (at == j * 32 + lane) key[j] = 0u;
        if (lane == k) id = at;
    }
    // the scores of the chosen, one lane each
    float mine = lane < m.top_k ? score(logits[id]) : 0.0f;
    const float sum = warp_sum(mine);
    if (lane < m.top_k) {
        if (m.renormalize) mine /= sum;
        ids[lane] = id;
        weights[lane] = mine * m.scale;
    }
}

cudaError_t launch_moe_plain(const MoeParams& m, int dtype, cudaStream_t s);
size_t moe_plain_workspace(int64_t tokens, int64_t inter, int experts, int top_k);
// The tensor-core form; false where its tensor maps do not apply.
bool launch_moe_tensor(const MoeParams& m, int dtype, cudaStream_t s, cudaError_t* e);
size_t moe_tensor_workspace(int64_t tokens, int64_t hidden, int64_t inter, int experts, int top_k);

}  // namespace ptoc
