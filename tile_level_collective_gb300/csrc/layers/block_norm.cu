// The norms around a block in one pass: rank-order sum of the N parts, norm
// after the block, gate, residual add, norm before the next block, and the
// 8-bit checkpoints of the block output and of the stream.
//
// Bound by HBM: N + 1 reads and 2 writes per element (plus 33/32 bytes for
// each checkpoint); the parameters stay in the caches. One block holds one
// row in registers (C chunks of 8 columns per thread), so each element is
// read once although two statistics of the row come before its last use.
#include "layers/layers_common.cuh"
#include "layers/layers_internal.h"

namespace ptoc {

namespace {

constexpr int kPartsInFlight = 4;

template <class T, bool V, int C>
__global__ void __launch_bounds__(1024) block_norm_kernel(const NormParams p)
{
    pdl_enter();
    __shared__ float slots[2][32];
    int turn = 0;                           // block_sum's slots in turn
    const NormCommon& k = p.c;
    const Ckpt bc{p.block_ckpt.codes, p.block_ckpt.exps, p.block_ckpt.ld_codes, p.block_ckpt.ld_exps};
    const Ckpt sc{p.stream_ckpt.codes, p.stream_ckpt.exps, p.stream_ckpt.ld_codes, p.stream_ckpt.ld_exps};
    for (int64_t row = blockIdx.x; row < k.rows; row += gridDim.x) {
        float a[C][8];
        Raw8<T> x[C];
        uint32_t mask[C];
#pragma unroll
        for (int i = 0; i < C; ++i) {
            const int64_t c = (int64_t)i * blockDim.x + threadIdx.x;
            mask[i] = chunk_mask<V>(c, k.cols);
            x[i] = load8<T, V>((const T*)p.x + row * p.ld_x, c, mask[i]);
        }
        // the parts in rank order, a group of loads in flight at a time
        for (int r0 = 0; r0 < p.nparts; r0 += kPartsInFlight) {
#pragma unroll
            for (int i = 0; i < C; ++i) {
                const int64_t c = (int64_t)i * blockDim.x + threadIdx.x;
                Raw8<T> w[kPartsInFlight];
#pragma unroll
                for (int q = 0; q < kPartsInFlight; ++q)
                    if (r0 + q < p.nparts)
                        w[q] = load8<T, V>((const T*)p.part[r0 + q] + row * p.ld_part, c, mask[i]);
#pragma unroll
                for (int q = 0; q < kPartsInFlight; ++q)
                    if (r0 + q < p.nparts)
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            const float v = w[q].at(j);
                            a[i][j] = r0 + q == 0 ? v : __fadd_rn(a[i][j], v);
                        }
            }
        }

        float ra = 1.0f;
        if (k.post_norm) {
            float sum[1] = {0.0f};
#pragma unroll
            for (int i = 0; i < C; ++i)
#pragma unroll
                for (int j = 0; j < 8; ++j) sum[0] += a[i][j] * a[i][j];
            block_sum(sum, slots[turn]);
            turn ^= 1;
            ra = 1.0f / sqrtf(sum[0] * k.inv_cols + k.eps);
        }

        float sq[1] = {0.0f};
#pragma unroll
        for (int i = 0; i < C; ++i) {
            const int64_t c = (int64_t)i * blockDim.x + threadIdx.x;
            if (p.block_out) store8<T, V>((T*)p.block_out + row * p.ld_block, c, mask[i], a[i]);
            if (bc.codes) ckpt_store8<V>(bc, row, c, mask[i], a[i]);
            float w[8], g[8];
            load_param8<T, V>(k.post_norm ? k.post_weight : nullptr, k.param_f32, c, mask[i], w);
            if (k.gate_cs) {
                const char* base = (const char*)k.gate + row * k.gate_rs * (k.param_f32 ? 4 : (int)sizeof(T));
                load_param8<T, V>(base, k.param_f32, c, mask[i], g);
            } else {
                float one = 1.0f;
                if (k.gate) one = k.param_f32 ? ((const float*)k.gate)[row * k.gate_rs]
                                              : to_f32(((const T*)k.gate)[row * k.gate_rs]);
#pragma unroll
                for (int j = 0; j < 8; ++j) g[j] = one;
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float n = a[i][j] * ra * w[j];
                a[i][j] = k.residual_scale * x[i].at(j) + k.branch_scale * (g[j] * n);
                sq[0] += a[i][j] * a[i][j];
            }
            store8<T, V>((T*)p.out + row * p.ld_out, c, mask[i], a[i]);
            if (sc.codes) {
                float v[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) v[j] = to_f32(from_f32<T>(a[i][j]));
                ckpt_store8<V>(sc, row, c, mask[i], v);
            }
        }
        if (p.normed || p.rstd) {
            block_sum(sq, slots[turn]);
            turn ^= 1;
            const float r = 1.0f / sqrtf(sq[0] * k.inv_cols + k.eps);
            if (p.rstd && threadIdx.x == 0) {
                p.rstd[row] = ra;
                p.rstd[k.rows + row] = r;
            }
            if (p.normed) {
#pragma unroll
                for (int i = 0; i < C; ++i) {
                    const int64_t c = (int64_t)i * blockDim.x + threadIdx.x;
                    float w[8];
                    load_param8<T, V>(k.pre_weight, k.param_f32, c, mask[i], w);
#pragma unroll
                    for (int j = 0; j < 8; ++j) w[j] = a[i][j] * r * w[j];
                    store8<T, V>((T*)p.normed + row * p.ld_normed, c, mask[i], w);
                }
            }
        }
    }
}

template <class T, bool V>
cudaError_t launch(const NormParams& p, cudaStream_t s)
{
    const int64_t groups = (p.c.cols + 255) / 256;           // warps' worth of chunks
    const dim3 grid((unsigned)(p.c.rows < INT32_MAX ? p.c.rows : INT32_MAX));
    if (groups <= 32) return launch_kernel(block_norm_kernel<T, V, 1>, grid, (unsigned)groups * 32, 0, s, p);
    if (groups <= 64) return launch_kernel(block_norm_kernel<T, V, 2>, grid, (unsigned)((groups + 1) / 2) * 32, 0, s, p);
    return launch_kernel(block_norm_kernel<T, V, 4>, grid, (unsigned)((groups + 3) / 4) * 32, 0, s, p);
}

}  // namespace

cudaError_t launch_block_norm(const NormParams& p, int dtype, cudaStream_t s)
{
    switch (dtype) {
    case PTOC_F32: return p.c.vec ? launch<float, true>(p, s) : launch<float, false>(p, s);
    case PTOC_F16: return p.c.vec ? launch<__half, true>(p, s) : launch<__half, false>(p, s);
    default: return p.c.vec ? launch<__nv_bfloat16, true>(p, s) : launch<__nv_bfloat16, false>(p, s);
    }
}

}  // namespace ptoc
