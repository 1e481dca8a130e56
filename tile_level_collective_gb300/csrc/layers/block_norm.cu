// The norms around a block in one pass: rank-order sum of the N parts, norm
// after the block, gate, residual add, norm before the next block, and the
// 8-bit checkpoints of the block output and of the stream.
//
// Bound by HBM: N + 1 reads and 2 writes per element (plus 33/32 bytes for
// each checkpoint). A block holds one row in registers (C chunks of 8 columns
// per thread), so each element is read once although two statistics of the
// row come before its last use. Two block-wide sums per row leave the memory
// idle unless the next rows are already on their way: one wave of blocks
// walks the rows, and every thread keeps a queue of copies of its own columns
// (the parts and the residual of this row and the next ones) in shared memory.
#include "layers/layers_common.cuh"
#include "layers/layers_internal.h"

namespace ptoc {

namespace {

// What follows the sum of the parts, for one row in registers: a (the sum) and
// x (raw) of C chunks. gw is the weight of the norm after the block times
// branch_scale and the gate where that varies along the columns; `scale` is
// the rest. wpre is the weight of the norm before the next block.

template <class T>
__device__ __forceinline__ float gate_of_row(const NormCommon& k, int64_t row)
{
    if (!k.gate) return 1.0f;
    return k.param_f32 ? ((const float*)k.gate)[row * k.gate_rs] : to_f32(((const T*)k.gate)[row * k.gate_rs]);
}

// The columns' factor of the norm after the block.
template <class T, bool V>
__device__ __forceinline__ void column_factor(const NormCommon& k, int64_t row, int64_t c, uint32_t mask, float* gw)
{
    load_param8<T, V>(k.post_weight, k.param_f32, c, mask, gw);
    if (k.gate_cs) {
        float g[8];
        const char* base = (const char*)k.gate + row * k.gate_rs * (k.param_f32 ? 4 : (int)sizeof(T));
        load_param8<T, V>(base, k.param_f32, c, mask, g);
#pragma unroll
        for (int j = 0; j < 8; ++j) gw[j] *= k.branch_scale * g[j];
    }
}

// KEEP: the column factors are in gw and wpre for all rows; else they are
// loaded for each row.
template <class T, bool V, int C, bool KEEP>
__device__ __forceinline__ void finish_row(const NormParams& p, int64_t row, float (&a)[C][8], const Raw8<T> (&x)[C],
                                           const uint32_t (&mask)[C], const float (&gw)[KEEP ? C : 1][8],
                                           const float (&wpre)[KEEP ? C : 1][8], float (*slots)[32], int& turn)
{
    const NormCommon& k = p.c;
    const Ckpt bc{p.block_ckpt.codes, p.block_ckpt.exps, p.block_ckpt.ld_codes, p.block_ckpt.ld_exps};
    const Ckpt sc{p.stream_ckpt.codes, p.stream_ckpt.exps, p.stream_ckpt.ld_codes, p.stream_ckpt.ld_exps};
    const float row_gate = k.gate_cs ? 1.0f : k.branch_scale * gate_of_row<T>(k, row);
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
    const float scale = ra * row_gate;
    float sq[1] = {0.0f};
#pragma unroll
    for (int i = 0; i < C; ++i) {
        const int64_t c = (int64_t)i * blockDim.x + threadIdx.x;
        if (p.block_out) store8<T, V>((T*)p.block_out + row * p.ld_block, c, mask[i], a[i]);
        if (bc.codes) ckpt_store8<V>(bc, row, c, mask[i], a[i]);
        float w[8];
        if constexpr (!KEEP) column_factor<T, V>(k, row, c, mask[i], w);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            a[i][j] = k.residual_scale * x[i].at(j) + a[i][j] * scale * (KEEP ? gw[KEEP ? i : 0][j] : w[j]);
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
    if (!p.normed && !p.rstd) return;
    block_sum(sq, slots[turn]);
    turn ^= 1;
    const float r = 1.0f / sqrtf(sq[0] * k.inv_cols + k.eps);
    if (p.rstd && threadIdx.x == 0) {
        p.rstd[row] = ra;
        p.rstd[k.rows + row] = r;
    }
    if (!p.normed) return;
#pragma unroll
    for (int i = 0; i < C; ++i) {
        const int64_t c = (int64_t)i * blockDim.x + threadIdx.x;
        float w[8];
        if constexpr (!KEEP) load_param8<T, V>(k.pre_weight, k.param_f32, c, mask[i], w);
#pragma unroll
        for (int j = 0; j < 8; ++j) w[j] = a[i][j] * r * (KEEP ? wpre[KEEP ? i : 0][j] : w[j]);
        store8<T, V>((T*)p.normed + row * p.ld_normed, c, mask[i], w);
    }
}

// Rows of 16-byte aligned words, through the threads' queues of K items.
// COLUMNS: the column factors are kept in registers (they do not depend on
// the row, and two chunks leave room for them).
template <class T, int C, int K, bool KEEP>
__global__ void __launch_bounds__(C == 2 ? 512 : 1024) block_norm_queue_kernel(const NormParams p)
{
    pdl_enter();
    extern __shared__ __align__(16) unsigned char smem[];
    __shared__ float slots[2][32];
    int turn = 0;                           // block_sum's slots in turn
    const NormCommon& k = p.c;
    Queue<C, (int)sizeof(T) / 2, K> queue(smem);
    uint32_t mask[C];
    float gw[KEEP ? C : 1][8], wpre[KEEP ? C : 1][8];
#pragma unroll
    for (int i = 0; i < C; ++i) {
        const int64_t c = (int64_t)i * blockDim.x + threadIdx.x;
        mask[i] = chunk_mask<true>(c, k.cols);
        if (!mask[i]) queue.clear(i);
    }
    // the item to copy next: source `src` (nparts: the residual) of row `ahead`
    int64_t ahead = blockIdx.x;
    int src = 0;
    auto push = [&] {
        if (ahead < k.rows) {
            const T* row = src < p.nparts ? (const T*)p.part[src] + ahead * p.ld_part : (const T*)p.x + ahead * p.ld_x;
            queue.template copy_row<T>(row, mask);
            if (++src > p.nparts) src = 0, ahead += gridDim.x;
        }
        queue.next();
    };
#pragma unroll 1
    for (int q = 0; q < K; ++q) push();
    if constexpr (KEEP)
#pragma unroll
        for (int i = 0; i < C; ++i) {
            const int64_t c = (int64_t)i * blockDim.x + threadIdx.x;
            column_factor<T, true>(k, 0, c, mask[i], gw[i]);
            load_param8<T, true>(k.pre_weight, k.param_f32, c, mask[i], wpre[i]);
        }
    for (int64_t row = blockIdx.x; row < k.rows; row += gridDim.x) {
        float a[C][8];
        Raw8<T> x[C];
        for (int r = 0; r < p.nparts; ++r) {
            queue.wait();
#pragma unroll
            for (int i = 0; i < C; ++i) {
                const Raw8<T> w = queue.template chunk<T>(i);
#pragma unroll
                for (int j = 0; j < 8; ++j) a[i][j] = r == 0 ? w.at(j) : __fadd_rn(a[i][j], w.at(j));
            }
            push();
        }
        queue.wait();
#pragma unroll
        for (int i = 0; i < C; ++i) x[i] = queue.template chunk<T>(i);
        push();
        finish_row<T, true, C, KEEP>(p, row, a, x, mask, gw, wpre, slots, turn);
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
}

// Rows at any address: element-wide accesses, the next row's by other blocks.
template <class T, int C>
__global__ void __launch_bounds__(1024) block_norm_kernel(const NormParams p)
{
    pdl_enter();
    __shared__ float slots[2][32];
    int turn = 0;
    const NormCommon& k = p.c;
    uint32_t mask[C];
#pragma unroll
    for (int i = 0; i < C; ++i) mask[i] = chunk_mask<false>((int64_t)i * blockDim.x + threadIdx.x, k.cols);
    for (int64_t row = blockIdx.x; row < k.rows; row += gridDim.x) {
        float a[C][8];
        Raw8<T> x[C];
#pragma unroll
        for (int i = 0; i < C; ++i)
            x[i] = load8<T, false>((const T*)p.x + row * p.ld_x, (int64_t)i * blockDim.x + threadIdx.x, mask[i]);
        for (int r = 0; r < p.nparts; ++r) {
            Raw8<T> w[C];
#pragma unroll
            for (int i = 0; i < C; ++i)
                w[i] = load8<T, false>((const T*)p.part[r] + row * p.ld_part, (int64_t)i * blockDim.x + threadIdx.x,
                                       mask[i]);
#pragma unroll
            for (int i = 0; i < C; ++i)
#pragma unroll
                for (int j = 0; j < 8; ++j) a[i][j] = r == 0 ? w[i].at(j) : __fadd_rn(a[i][j], w[i].at(j));
        }
        const float none[1][8] = {};
        finish_row<T, false, C, false>(p, row, a, x, mask, none, none, slots, turn);
    }
}

template <class T, int C, int K>
cudaError_t launch_queue(const NormParams& p, cudaStream_t s)
{
    const int64_t chunks = p.c.cols / 8;
    const unsigned threads = (unsigned)((chunks + 32 * C - 1) / (32 * C)) * 32;
    const size_t smem = (size_t)K * threads * C * sizeof(T) * 8;
    // one wave: the registers and the queues of 512 threads of two chunks fill an SM
    const int64_t per_sm = C == 2 ? (512 / threads < 16 ? 512 / threads : 16) : 1;
    const int64_t most = 152 * per_sm;
    const dim3 grid((unsigned)(p.c.rows < most ? p.c.rows : most));
    const bool keep = C == 2 && !(p.c.gate_cs && p.c.gate_rs);
    auto kernel = keep ? block_norm_queue_kernel<T, C, K, C == 2> : block_norm_queue_kernel<T, C, K, false>;
    const cudaError_t e = cudaFuncSetAttribute((const void*)kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               (int)(K * (C == 2 ? 512 : 1024) * C * sizeof(T) * 8));
    if (e != cudaSuccess) return e;
    return launch_kernel(kernel, grid, threads, smem, s, p);
}

template <class T>
cudaError_t launch(const NormParams& p, cudaStream_t s)
{
    constexpr int kItems = 12 / ((int)sizeof(T) / 2);        // 192 KiB of queues on an SM
    if (p.c.vec) {
        if (p.c.cols <= 8192) return launch_queue<T, 2, kItems>(p, s);
        return launch_queue<T, 4, kItems / 4>(p, s);
    }
    const int64_t groups = (p.c.cols + 255) / 256;           // warps' worth of chunks
    const dim3 grid((unsigned)(p.c.rows < INT32_MAX ? p.c.rows : INT32_MAX));
    if (groups <= 32) return launch_kernel(block_norm_kernel<T, 1>, grid, (unsigned)groups * 32, 0, s, p);
    if (groups <= 64) return launch_kernel(block_norm_kernel<T, 2>, grid, (unsigned)((groups + 1) / 2) * 32, 0, s, p);
    return launch_kernel(block_norm_kernel<T, 4>, grid, (unsigned)((groups + 3) / 4) * 32, 0, s, p);
}

}  // namespace

cudaError_t launch_block_norm(const NormParams& p, int dtype, cudaStream_t s)
{
    switch (dtype) {
    case PTOC_F32: return launch<float>(p, s);
    case PTOC_F16: return launch<__half>(p, s);
    default: return launch<__nv_bfloat16>(p, s);
    }
}

}  // namespace ptoc
