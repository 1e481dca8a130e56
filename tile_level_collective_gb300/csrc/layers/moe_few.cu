// A mixture-of-experts layer for a few tokens, in its plain form, for rows
// that the tensor-core form's copies cannot address: router dot products, the
// choice, the gated first product and the weighted second one, one launch
// each, a warp per output row.
//
// At one token bound by its loads of one element per lane: the chosen experts'
// 3 * inter * hidden weights pass once, at a quarter of the copy rate. With more
// tokens they pass more often: the first product reads a gate and an up row
// once for every eight pairs of its expert, the second one a row of the output
// weights once for every token that chose the expert.
//
// Measured on GB300 (bf16, weights at an odd element): 1 token, 8 of 64 experts
// of 7168 x 2048, 440 us (floor 104 at 6.79 TB/s); 13 tokens of 16 experts of
// 4096 x 1536 860 us (floor 83), 64 tokens 3,920 us (floor 89; the tensor-core
// form at aligned rows 148).
#include "layers/moe_common.cuh"

namespace ptoc {

namespace {

constexpr int kWarps = kBlock / 32;
constexpr int kTokensAtOnce = 8;

struct MoePlan {
    float* logits;                // [tokens, experts]
    int32_t* ids;                 // [tokens, top_k]
    float* weights;               // [tokens, top_k]
    float* hidden;                // [tokens * top_k, inter] activations, weighted
};

constexpr size_t align256(size_t n) { return (n + 255) / 256 * 256; }

size_t plan_bytes(int64_t tokens, int64_t inter, int experts, int top_k, size_t off[4])
{
    size_t at = 0;
    off[0] = at, at += align256((size_t)tokens * experts * 4);
    off[1] = at, at += align256((size_t)tokens * top_k * 4);
    off[2] = at, at += align256((size_t)tokens * top_k * 4);
    off[3] = at, at += align256((size_t)tokens * top_k * inter * 4);
    return at;
}

struct MoePlainParams {
    MoeParams m;
    MoePlan w;
};

template <class T>
__device__ __forceinline__ float param_at(const void* p, bool f32, int64_t i)
{
    return f32 ? ((const float*)p)[i] : to_f32(((const T*)p)[i]);
}

template <class T>
__global__ void __launch_bounds__(kBlock) moe_router_kernel(const MoePlainParams p)
{
    pdl_enter();
    const int lane = threadIdx.x & 31;
    const int dot = blockIdx.x * kWarps + (threadIdx.x >> 5);
    if (dot >= p.m.tokens * p.m.experts) return;
    const int t = dot / p.m.experts, e = dot - t * p.m.experts;
    const T* x = (const T*)p.m.x + t * p.m.ld_x;
    const int64_t r = (int64_t)e * p.m.hidden;
    float sum = 0.0f;
#pragma unroll 4
    for (int64_t h = lane; h < p.m.hidden; h += 32)
        sum += to_f32(x[h]) * param_at<T>(p.m.router, p.m.router_f32, r + h);
    sum = warp_sum(sum);
    if (lane == 0) p.w.logits[dot] = sum;
}

// One warp per token.
template <int L>
__global__ void __launch_bounds__(32) moe_choose_kernel(const MoePlainParams p)
{
    pdl_enter();
    const int t = blockIdx.x, i = t * p.m.top_k + threadIdx.x;
    int32_t* ids = p.w.ids + t * p.m.top_k;
    choose_experts<L>(p.m, p.w.logits + (int64_t)t * p.m.experts, ids, p.w.weights + t * p.m.top_k);
    __syncwarp();
    if (threadIdx.x < p.m.top_k) {
        if (p.m.ids) p.m.ids[i] = p.w.ids[i];
        if (p.m.weights) p.m.weights[i] = p.w.weights[i];
    }
}

// A warp takes row i of one local expert's gate and up weights.
template <class T>
__global__ void __launch_bounds__(kBlock) moe_in_kernel(const MoePlainParams p)
{
    pdl_enter();
    __shared__ int16_t list[PTOC_MOE_MAX_TOKENS];
    __shared__ int count;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int local = blockIdx.y, pairs = p.m.tokens * p.m.top_k;
    if (warp == 0) {
        int n = 0;
        for (int q0 = 0; q0 < pairs; q0 += 32) {
            const bool hit = q0 + lane < pairs && p.w.ids[q0 + lane] == p.m.first + local;
            const uint32_t m = __ballot_sync(0xffffffffu, hit);
            if (hit) list[n + __popc(m & ((1u << lane) - 1))] = (int16_t)(q0 + lane);
            n += __popc(m);
        }
        if (lane == 0) count = n;
    }
    __syncthreads();
    const int64_t i = (int64_t)blockIdx.x * kWarps + warp, h = p.m.hidden;
    if (i >= p.m.inter) return;
    const T* wg = (const T*)p.m.w_in + ((int64_t)local * 2 * p.m.inter + i) * h;
    const T* wu = wg + p.m.inter * h;
    for (int q0 = 0; q0 < count; q0 += kTokensAtOnce) {
        const T* x[kTokensAtOnce];
        float g[kTokensAtOnce] = {}, u[kTokensAtOnce] = {};
#pragma unroll
        for (int q = 0; q < kTokensAtOnce; ++q)
            x[q] = (const T*)p.m.x + list[min(q0 + q, count - 1)] / p.m.top_k * p.m.ld_x;
        for (int64_t c = lane; c < h; c += 32) {
            const float a = to_f32(wg[c]), b = to_f32(wu[c]);
#pragma unroll
            for (int q = 0; q < kTokensAtOnce; ++q) {
                if (q0 + q >= count) break;
                const float v = to_f32(x[q][c]);
                g[q] += a * v;
                u[q] += b * v;
            }
        }
#pragma unroll
        for (int q = 0; q < kTokensAtOnce; ++q) {
            if (q0 + q >= count) break;
            const float gs = warp_sum(g[q]), us = warp_sum(u[q]);
            const int pair = list[q0 + q];
            if (lane == 0)
                p.w.hidden[pair * p.m.inter + i] =
                    split_parts<T>(p.w.weights[pair] * (gs / (1.0f + expf(-gs)) * us)).value();
        }
    }
}

// A warp takes column h of the output for every token.
template <class T>
__global__ void __launch_bounds__(kBlock) moe_out_kernel(const MoePlainParams p)
{
    pdl_enter();
    const int lane = threadIdx.x & 31;
    const int64_t h = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5), n = p.m.inter;
    if (h >= p.m.hidden) return;
    for (int t = 0; t < p.m.tokens; ++t) {
        float sum = 0.0f;
        for (int k = 0; k < p.m.top_k; ++k) {
            const int pair = t * p.m.top_k + k, local = p.w.ids[pair] - p.m.first;
            if (local < 0 || local >= p.m.local) continue;
            const T* w = (const T*)p.m.w_out + ((int64_t)local * p.m.hidden + h) * n;
            const float* act = p.w.hidden + pair * n;
#pragma unroll 4
            for (int64_t c = lane; c < n; c += 32) sum += to_f32(w[c]) * act[c];
        }
        sum = warp_sum(sum);
        if (lane == 0) ((T*)p.m.y)[t * p.m.ld_y + h] = from_f32<T>(sum);
    }
}

template <class T>
cudaError_t launch_plain(const MoePlainParams& p, cudaStream_t s)
{
    const int dots = p.m.tokens * p.m.experts;
    cudaError_t e = launch_kernel(moe_router_kernel<T>, dim3((dots + kWarps - 1) / kWarps), kBlock, 0, s, p);
    if (e == cudaSuccess)
        e = p.m.experts <= 128 ? launch_kernel(moe_choose_kernel<4>, dim3(p.m.tokens), 32, 0, s, p)
                               : launch_kernel(moe_choose_kernel<32>, dim3(p.m.tokens), 32, 0, s, p);
    const dim3 in((unsigned)((p.m.inter + kWarps - 1) / kWarps), p.m.local);
    if (e == cudaSuccess) e = launch_kernel(moe_in_kernel<T>, in, kBlock, 0, s, p);
    const dim3 out((unsigned)((p.m.hidden + kWarps - 1) / kWarps));
    if (e == cudaSuccess) e = launch_kernel(moe_out_kernel<T>, out, kBlock, 0, s, p);
    return e;
}

}  // namespace

size_t moe_plain_workspace(int64_t tokens, int64_t inter, int experts, int top_k)
{
    size_t off[4];
    return plan_bytes(tokens, inter, experts, top_k, off);
}

cudaError_t launch_moe_plain(const MoeParams& m, int dtype, cudaStream_t s)
{
    size_t off[4];
    plan_bytes(m.tokens, m.inter, m.experts, m.top_k, off);
    MoePlainParams p{m, MoePlan{(float*)(m.ws + off[0]), (int32_t*)(m.ws + off[1]), (float*)(m.ws + off[2]),
                                (float*)(m.ws + off[3])}};
    return dtype == PTOC_F16 ? launch_plain<__half>(p, s) : launch_plain<__nv_bfloat16>(p, s);
}

size_t moe_workspace_bytes(int64_t tokens, int64_t hidden, int64_t inter, int experts, int top_k)
{
    const size_t a = moe_plain_workspace(tokens, inter, experts, top_k);
    const size_t b = moe_tensor_workspace(tokens, hidden, inter, experts, top_k);
    return a > b ? a : b;
}

cudaError_t launch_moe_few(const MoeParams& m, int dtype, cudaStream_t s)
{
    cudaError_t e = cudaSuccess;
    if (m.vec && launch_moe_tensor(m, dtype, s, &e)) return e;
    return launch_moe_plain(m, dtype, s);
}

}  // namespace ptoc
