// The backward pass of the norms around a block.
//
// Bound by HBM: per element it reads dy, du, s and a (the last two in 2 or 4
// bytes, or 33/32 as 8-bit checkpoints) and writes d_residual and d_block.
// One wave of blocks walks the rows; a thread keeps the sums over its rows of
// its columns' weight and gate gradients in registers. Each block writes them
// as one partial row, and a second launch adds the partial rows in order.
#include "layers/layers_common.cuh"
#include "layers/layers_internal.h"

namespace ptoc {

namespace {

template <class T, bool V>
__device__ __forceinline__ void load_saved8(const void* m, int64_t ld, const Ckpt& k, int64_t row, int64_t c,
                                            uint32_t mask, float* v)
{
    if (m) {
        const Raw8<T> r = load8<T, V>((const T*)m + row * ld, c, mask);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = r.at(j);
    } else {
        ckpt_load8<V>(k, row, c, mask, v);
    }
}

template <class T, bool V, int C>
__global__ void __launch_bounds__(1024) norm_backward_kernel(const NormBackParams p)
{
    pdl_enter();
    __shared__ float slots[2][2 * 32];
    int turn = 0;                           // block_sum's slots in turn
    const NormCommon& k = p.c;
    const Ckpt bc{p.block_ckpt.codes, p.block_ckpt.exps, p.block_ckpt.ld_codes, p.block_ckpt.ld_exps};
    const Ckpt sc{p.stream_ckpt.codes, p.stream_ckpt.exps, p.stream_ckpt.ld_codes, p.stream_ckpt.ld_exps};
    float sum_pre[C][8] = {}, sum_post[C][8] = {}, sum_gate[C][8] = {};
    float sum_scalar = 0.0f;
    for (int64_t row = blockIdx.x; row < k.rows; row += gridDim.x) {
        const float ra = k.post_norm ? p.rstd[row] : 1.0f, r = p.rstd[k.rows + row];
        float st[C][8], up[C][8], a[C][8];
        float dot[1] = {0.0f};
#pragma unroll
        for (int i = 0; i < C; ++i) {
            const int64_t c = (int64_t)i * blockDim.x + threadIdx.x;
            const uint32_t mask = chunk_mask<V>(c, k.cols);
            load_saved8<T, V>(p.stream, p.ld_stream, sc, row, c, mask, st[i]);
            load_saved8<T, V>(p.block, p.ld_block, bc, row, c, mask, a[i]);
            const Raw8<T> dy = load8<T, V>((const T*)p.dy + row * p.ld_dy, c, mask);
            float w[8];
            load_param8<T, V>(k.pre_weight, k.param_f32, c, mask, w);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                st[i][j] *= r;
                up[i][j] = w[j] * dy.at(j);
                sum_pre[i][j] += dy.at(j) * st[i][j];
                dot[0] += up[i][j] * st[i][j];
            }
        }
        block_sum(dot, slots[turn]);
        turn ^= 1;
        const float m = dot[0] * k.inv_cols;
        // up becomes dn (times the weight of the norm after), a becomes a * ra
        float dots[2] = {0.0f, 0.0f};
#pragma unroll
        for (int i = 0; i < C; ++i) {
            const int64_t c = (int64_t)i * blockDim.x + threadIdx.x;
            const uint32_t mask = chunk_mask<V>(c, k.cols);
            float ds[8], w[8], g[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) ds[j] = r * (up[i][j] - m * st[i][j]);
            if (p.du) {
                const Raw8<T> du = load8<T, V>((const T*)p.du + row * p.ld_du, c, mask);
#pragma unroll
                for (int j = 0; j < 8; ++j) ds[j] += du.at(j);
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) w[j] = k.residual_scale * ds[j];
            store8<T, V>((T*)p.d_residual + row * p.ld_dres, c, mask, w);
            load_param8<T, V>(k.post_norm ? k.post_weight : nullptr, k.param_f32, c, mask, w);
            if (k.gate_cs) {
                const char* base = (const char*)k.gate + row * k.gate_rs * (k.param_f32 ? 4 : (int)sizeof(T));
                load_param8<T, V>(base, k.param_f32, c, mask, g);
            } else {
                float one = 1.0f;
                if (k.gate) one = k.param_f32 ? ((const float*)k.gate)[row * k.gate_rs]
                                              : to_f32(((const T*)k.gate)[row * k.gate_rs]);
#pragma unroll
                for (int j = 0; j < 8; ++j) g[j] = one;
            }
            float dg[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                a[i][j] *= ra;
                const float dn = k.branch_scale * (g[j] * ds[j]);
                dg[j] = k.branch_scale * (ds[j] * (a[i][j] * w[j]));
                sum_post[i][j] += dn * a[i][j];
                up[i][j] = dn * w[j];
                dots[0] += up[i][j] * a[i][j];
                dots[1] += dg[j];
                sum_gate[i][j] += dg[j];
            }
            if (p.gate_kind == kGateElement) {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (mask >> j & 1) p.d_gate[row * k.cols + col_of<V>(c, j)] = dg[j];
            }
        }
        if (k.post_norm || p.gate_kind == kGateToken || p.gate_kind == kGateScalar) {
            block_sum(dots, slots[turn]);
            turn ^= 1;
        }
        const float m2 = k.post_norm ? dots[0] * k.inv_cols : 0.0f;
        if (p.gate_kind == kGateToken && threadIdx.x == 0) p.d_gate[row] = dots[1];
        sum_scalar += dots[1];
#pragma unroll
        for (int i = 0; i < C; ++i) {
            const int64_t c = (int64_t)i * blockDim.x + threadIdx.x;
            float v[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = ra * (up[i][j] - m2 * a[i][j]);
            store8<T, V>((T*)p.d_block + row * p.ld_dblk, c, chunk_mask<V>(c, k.cols), v);
        }
    }
    // this block's partial rows
    const int64_t plane = (int64_t)gridDim.x * k.cols;
    float* mine = p.partial + (int64_t)blockIdx.x * k.cols;
#pragma unroll
    for (int i = 0; i < C; ++i) {
        const int64_t c = (int64_t)i * blockDim.x + threadIdx.x;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int64_t col = col_of<V>(c, j);
            if (col >= k.cols) continue;
            if (p.d_pre) mine[col] = sum_pre[i][j];
            if (p.d_post) mine[plane + col] = sum_post[i][j];
            if (p.gate_kind == kGateChannel) mine[2 * plane + col] = sum_gate[i][j];
        }
    }
    if (p.gate_kind == kGateScalar && threadIdx.x == 0) mine[2 * plane] = sum_scalar;
}

// Sums of the partial rows: a block takes 32 columns of one kind; its 8 warps
// each add a run of the partial rows in order, and the runs are added in order.
__global__ void __launch_bounds__(kBlock) norm_backward_sum_kernel(const NormBackParams p)
{
    pdl_enter();
    __shared__ float runs[kBlock / 32][32];
    const int64_t cols = p.c.cols, plane = (int64_t)p.grid * cols;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t col = (int64_t)blockIdx.x * 32 + lane;
    const int kind = blockIdx.y;
    float* dst = kind == 0 ? p.d_pre : kind == 1 ? p.d_post : p.d_gate;
    const int64_t n = kind < 2 ? cols : p.gate_kind == kGateChannel ? cols : p.gate_kind == kGateScalar ? 1 : 0;
    const bool live = dst && col < n;
    float sum = 0.0f;
    if (live) {
        const float* src = p.partial + kind * plane + col;
        const int per = (p.grid + kBlock / 32 - 1) / (kBlock / 32);
        const int end = min(p.grid, (warp + 1) * per);
#pragma unroll 8
        for (int b = warp * per; b < end; ++b) sum += src[(int64_t)b * cols];
    }
    runs[warp][lane] = sum;
    __syncthreads();
    if (warp == 0 && live) {
        sum = 0.0f;
#pragma unroll
        for (int w = 0; w < kBlock / 32; ++w) sum += runs[w][lane];
        dst[col] = sum;
    }
}

template <class T, bool V>
cudaError_t launch(const NormBackParams& p, cudaStream_t s)
{
    const int64_t groups = (p.c.cols + 255) / 256;
    const dim3 grid((unsigned)p.grid);
    if (groups <= 32) return launch_kernel(norm_backward_kernel<T, V, 1>, grid, (unsigned)groups * 32, 0, s, p);
    if (groups <= 64)
        return launch_kernel(norm_backward_kernel<T, V, 2>, grid, (unsigned)((groups + 1) / 2) * 32, 0, s, p);
    return launch_kernel(norm_backward_kernel<T, V, 4>, grid, (unsigned)((groups + 3) / 4) * 32, 0, s, p);
}

}  // namespace

// Rows of up to 2048 columns leave room for several blocks on an SM. The
// count is GB300's, not the device's answer: the order of the sums and the
// workspace then depend on the sizes alone.
int norm_backward_grid(int64_t rows, int64_t cols)
{
    constexpr int kSms = 152;
    const int per_sm = cols <= 2048 ? 4 : cols <= 4096 ? 2 : 1;
    const int64_t most = (int64_t)kSms * per_sm;
    return (int)(rows < most ? rows : most);
}

cudaError_t launch_block_norm_backward(const NormBackParams& p, int dtype, cudaStream_t s)
{
    cudaError_t e;
    switch (dtype) {
    case PTOC_F32: e = p.c.vec ? launch<float, true>(p, s) : launch<float, false>(p, s); break;
    case PTOC_F16: e = p.c.vec ? launch<__half, true>(p, s) : launch<__half, false>(p, s); break;
    default: e = p.c.vec ? launch<__nv_bfloat16, true>(p, s) : launch<__nv_bfloat16, false>(p, s); break;
    }
    if (e != cudaSuccess) return e;
    const bool gate_sum = p.gate_kind == kGateChannel || p.gate_kind == kGateScalar;
    if (!p.d_pre && !p.d_post && !gate_sum) return cudaSuccess;
    const dim3 grid((unsigned)((p.c.cols + 31) / 32), kNormColumnSums);
    return launch_kernel(norm_backward_sum_kernel, grid, kBlock, 0, s, p);
}

}  // namespace ptoc
