// The norms around a block in one pass: rank-order sum of the N parts, norm
// after the block, gate, residual add, norm before the next block, and the
// 8-bit checkpoints of the block output and of the stream.
//
// Bound by HBM: N + 1 reads and 2 writes per element (plus 33/32 bytes for
// each checkpoint). A block holds one row in registers (C chunks of 8 columns
// per thread), so each element is read once although two statistics of the
// row come before its last use. Two block-wide sums per row leave the memory
// idle unless the next rows are already on their way: one wave of blocks
// walks the rows, and every warp keeps a queue of copies of its own columns
// (the parts and the residual of this row and the next ones) in shared memory.
// That holds up to 8,192 columns. Wider rows take four chunks per thread in 64
// registers, some of them spilled, and queues of three items (16-bit types) or
// one (binary32, which is waited for at once).
//
// Measured on GB300 (bf16; of 6.79 TB/s copied): 16384 x 8192 of 8 parts 436 us
// (6.8 TB/s; one block per row without a queue: 650 us); of 1 part 167 us (6.4
// TB/s), with both checkpoints 212 us (6.4 TB/s); 8192 x 4096 of 1 part 46 us (5.8
// TB/s), with both checkpoints 58 us (5.8 TB/s: 36 million instructions, 58 % of
// the issue slots at 16 warps per SM), of 4095 columns 110 us (8 accesses where
// an aligned row takes one). Wide rows of 1 part with both checkpoints: 5461 x
// 12288 263 us and 2048 x 32768 171 us (floor 99; 8192 x 8192 takes 111). One row
// of 7168 columns of 8 parts: 4.9 us on the device.
#include "layers/layers_common.cuh"
#include "layers/layers_internal.h"

namespace ptoc {

namespace {

template <class T>
__device__ __forceinline__ float gate_of_row(const NormCommon& k, int64_t row)
{
    if (!k.gate || k.gate_cs) return 1.0f;
    return k.param_f32 ? ((const float*)k.gate)[row * k.gate_rs] : to_f32(((const T*)k.gate)[row * k.gate_rs]);
}

// The columns' factor of the norm after the block: its weight, times
// branch_scale * gate where the gate varies along the columns.
template <class T, int G>
__device__ __forceinline__ F8 column_factor(const NormCommon& k, int64_t row, int32_t col, uint32_t mask)
{
    F8 w = load_param8<T, G>(k.post_weight, k.param_f32, col, mask);
    if (k.gate_cs) {
        const char* base = (const char*)k.gate + row * k.gate_rs * (k.param_f32 ? 4 : (int)sizeof(T));
        const F8 g = load_param8<T, G>(base, k.param_f32, col, mask);
#pragma unroll
        for (int j = 0; j < 4; ++j) w.p[j] = mul2(w.p[j], mul2(both(k.branch_scale), g.p[j]));
    }
    return w;
}

template <int C>
__device__ __forceinline__ float square_sum(const F8 (&a)[C])
{
    Pair sum[2 * C];                        // (short chains of dependent operations)
#pragma unroll
    for (int i = 0; i < 2 * C; ++i) {
        const Pair u = a[i / 2].p[2 * (i & 1)], v = a[i / 2].p[2 * (i & 1) + 1];
        sum[i] = fma2(u, u, mul2(v, v));
    }
#pragma unroll
    for (int n = C; n > 0; n /= 2)
#pragma unroll
        for (int i = 0; i < n; ++i) sum[i] = add2(sum[i], sum[i + n]);
    return sum_of(sum[0]);
}

// What follows the sum of the parts, for one row in registers: a (the sum) and
// x of C chunks. KEEP: the column factors are in gw and wpre for all rows;
// else they are loaded for each row. FULL: a norm after the block, both
// checkpoints and `normed`, but no matrix of the block output are asked for.
template <class T, int G, int C, bool KEEP, bool FULL = false>
__device__ __forceinline__ void finish_row(const NormParams& p, int64_t row, F8 (&a)[C], const Raw8<T, G> (&x)[C],
                                           const int32_t (&col)[C], const uint32_t (&mask)[C],
                                           const F8 (&gw)[KEEP ? C : 1], const F8 (&wpre)[KEEP ? C : 1],
                                           float gate, SumSlots<1>& sums)
{
    const NormCommon& k = p.c;
    const Ckpt bc{p.block_ckpt.codes, p.block_ckpt.exps, p.block_ckpt.ld_codes, p.block_ckpt.ld_exps};
    const Ckpt sc{p.stream_ckpt.codes, p.stream_ckpt.exps, p.stream_ckpt.ld_codes, p.stream_ckpt.ld_exps};
    const float row_gate = k.gate_cs ? 1.0f : k.branch_scale * gate;
    float ra = 1.0f, total[1];
    if (FULL || k.post_norm) {
        total[0] = square_sum(a);
        sums.begin(total);
    }
    if (!FULL && p.block_out)
#pragma unroll
        for (int i = 0; i < C; ++i) store8<T, G>((T*)p.block_out + row * p.ld_block, col[i], mask[i], a[i]);
    if (FULL || bc.codes)
#pragma unroll
        for (int i = 0; i < C; ++i) ckpt_store8<G>(bc, row, col[0], i, mask[i], a[i]);
    if (FULL || k.post_norm) {
        sums.end(total);
        ra = 1.0f / sqrtf(total[0] * k.inv_cols + k.eps);
    }
    // (past the row's end 0 times a factor that is not finite would be NaN)
    const float scale = ra * row_gate;
    Raw8<T, G> s[C];
#pragma unroll
    for (int i = 0; i < C; ++i) {
        F8 w;
        if constexpr (!KEEP) w = column_factor<T, G>(k, row, col[i], mask[i]);
        const F8 r = x[i].expand();
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const bool lo = mask[i] >> (2 * j / G) & 1, hi = mask[i] >> ((2 * j + 1) / G) & 1;
            const Pair scales = pair(lo ? scale : 0.0f, hi ? scale : 0.0f);
            const Pair keep = pair(lo ? k.residual_scale : 0.0f, hi ? k.residual_scale : 0.0f);
            const Pair n = mul2(mul2(a[i].p[j], scales), KEEP ? gw[KEEP ? i : 0].p[j] : w.p[j]);
            a[i].p[j] = fma2(keep, r.p[j], n);
        }
        s[i] = round8<T, G>(a[i]);
        store8<T, G>((T*)p.out + row * p.ld_out, col[i], mask[i], s[i]);
    }
    const bool statistic = FULL || p.normed || p.rstd;
    if (statistic) {
        total[0] = square_sum(a);
        sums.begin(total);
    }
    if (FULL || sc.codes)
#pragma unroll
        for (int i = 0; i < C; ++i) ckpt_store8<G>(sc, row, col[0], i, mask[i], s[i].expand());
    if (!statistic) return;
    sums.end(total);
    const float r = 1.0f / sqrtf(total[0] * k.inv_cols + k.eps);
    if (p.rstd && threadIdx.x == 0) {
        p.rstd[row] = ra;
        p.rstd[k.rows + row] = r;
    }
    if (!FULL && !p.normed) return;
#pragma unroll
    for (int i = 0; i < C; ++i) {
        F8 w;
        if constexpr (!KEEP) w = load_param8<T, G>(k.pre_weight, k.param_f32, col[i], mask[i]);
#pragma unroll
        for (int j = 0; j < 4; ++j) a[i].p[j] = mul2(mul2(a[i].p[j], both(r)), KEEP ? wpre[KEEP ? i : 0].p[j] : w.p[j]);
        store8<T, G>((T*)p.normed + row * p.ld_normed, col[i], mask[i], a[i]);
    }
}

// Through the warps' queues of K items. KEEP: the column factors stay in
// registers (they do not depend on the row, and two chunks leave room for them).
// The bound of one block per SM keeps the compiler from saving registers that
// nothing else would use: 8192 x 4096 with both checkpoints takes 58 us with 105
// registers, and took 70 with 82 where 95 took 58.
template <class T, int C, int K, bool KEEP, bool ODD, bool FULL = false>
__global__ void __launch_bounds__(C == 2 ? 512 : 1024, 1) block_norm_queue_kernel(const NormParams p)
{
    constexpr int G = ODD ? 1 : kVector<T>;
    pdl_enter();
    extern __shared__ __align__(16) unsigned char smem[];
    __shared__ __align__(16) float slots[2 * 32];
    SumSlots<1> sums(slots);
    const NormCommon& k = p.c;
    int32_t col[C];
    uint32_t mask[C];
    F8 gw[KEEP ? C : 1], wpre[KEEP ? C : 1];
#pragma unroll
    for (int i = 0; i < C; ++i) {
        col[i] = first_col<G, C>(i);
        mask[i] = runs_below<G>(col[i], k.cols);
    }
    Queue<T, C, K, ODD> queue(smem, mask);
    // the item to copy next: source `src` (nparts: the residual) of row `ahead`
    int64_t ahead = blockIdx.x, part_at = ahead * p.ld_part;
    const T* x_row = (const T*)p.x + ahead * p.ld_x;
    int src = 0;
    auto push = [&] {
        queue.done();
        if (ahead < k.rows) {
            if (src < p.nparts) {
                queue.copy_row((const T*)p.part[src] + part_at, col, mask, k.cols);
                ++src;
            } else {
                queue.copy_row(x_row, col, mask, k.cols);
                src = 0;
                ahead += gridDim.x;
                part_at += p.step_part;
                x_row += p.step_x;
            }
        }
        queue.next();
    };
#pragma unroll 1
    for (int q = 0; q < K; ++q) push();
    if constexpr (KEEP)
#pragma unroll
        for (int i = 0; i < C; ++i) {
            gw[i] = column_factor<T, G>(k, 0, col[i], mask[i]);
            wpre[i] = load_param8<T, G>(k.pre_weight, k.param_f32, col[i], mask[i]);
        }
    // the row's gate (where it is one number), read a row before its use
    float gate = gate_of_row<T>(k, blockIdx.x);
    for (int64_t row = blockIdx.x; row < k.rows; row += gridDim.x) {
        const float next_gate = row + gridDim.x < k.rows ? gate_of_row<T>(k, row + gridDim.x) : 0.0f;
        // where the rows begin in their words
        const uint32_t part_shift = (uint32_t)row * (uint32_t)p.ld_part * (uint32_t)sizeof(T) & 15u;
        const uint32_t x_shift = (uint32_t)row * (uint32_t)p.ld_x * (uint32_t)sizeof(T) & 15u;
        F8 a[C];
        Raw8<T, G> x[C];
        queue.wait();
#pragma unroll
        for (int i = 0; i < C; ++i) a[i] = queue.chunk(i, part_shift).expand();
        push();
        for (int r = 1; r < p.nparts; ++r) {
            queue.wait();
#pragma unroll
            for (int i = 0; i < C; ++i) {
                const F8 w = queue.chunk(i, part_shift).expand();
#pragma unroll
                for (int j = 0; j < 4; ++j) a[i].p[j] = add2(a[i].p[j], w.p[j]);
            }
            push();
        }
        queue.wait();
#pragma unroll
        for (int i = 0; i < C; ++i) x[i] = queue.chunk(i, x_shift);
        push();
        finish_row<T, G, C, KEEP, FULL>(p, row, a, x, col, mask, gw, wpre, gate, sums);
        gate = next_gate;
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
}

// Rows whose base is not 16-byte aligned: element-wide accesses, the next row's
// by other blocks.
template <class T, int C>
__global__ void __launch_bounds__(C == 2 ? 512 : 1024) block_norm_kernel(const NormParams p)
{
    pdl_enter();
    __shared__ __align__(16) float slots[2 * 32];
    SumSlots<1> sums(slots);
    const NormCommon& k = p.c;
    int32_t col[C];
    uint32_t mask[C];
#pragma unroll
    for (int i = 0; i < C; ++i) {
        col[i] = first_col<1, C>(i);
        mask[i] = runs_below<1>(col[i], k.cols);
    }
    for (int64_t row = blockIdx.x; row < k.rows; row += gridDim.x) {
        F8 a[C];
        Raw8<T, 1> x[C];
#pragma unroll
        for (int i = 0; i < C; ++i) {
            x[i] = load8<T, 1>((const T*)p.x + row * p.ld_x, col[i], mask[i]);
            a[i] = load8<T, 1>((const T*)p.part[0] + row * p.ld_part, col[i], mask[i]).expand();
        }
        for (int r = 1; r < p.nparts; ++r) {
            Raw8<T, 1> w[C];
#pragma unroll
            for (int i = 0; i < C; ++i) w[i] = load8<T, 1>((const T*)p.part[r] + row * p.ld_part, col[i], mask[i]);
#pragma unroll
            for (int i = 0; i < C; ++i) {
                const F8 f = w[i].expand();
#pragma unroll
                for (int j = 0; j < 4; ++j) a[i].p[j] = add2(a[i].p[j], f.p[j]);
            }
        }
        const F8 none[1] = {};
        finish_row<T, 1, C, false>(p, row, a, x, col, mask, none, none, gate_of_row<T>(k, row), sums);
    }
}

template <class T, int C, int K, bool ODD>
cudaError_t launch_queue(const NormParams& p, cudaStream_t s)
{
    const int64_t groups = (p.c.cols + 255) / 256;           // warps' worth of chunks
    const unsigned threads = (unsigned)((groups + C - 1) / C) * 32;
    // one wave: the registers and the queues of 512 threads of two chunks fill an SM
    const int64_t per_sm = C == 2 ? (512 / threads < 16 ? 512 / threads : 16) : 1;
    const int64_t most = 152 * per_sm;
    const dim3 grid((unsigned)(p.c.rows < most ? p.c.rows : most));
    const bool keep = C == 2 && !(p.c.gate_cs && p.c.gate_rs);
    auto kernel = keep ? block_norm_queue_kernel<T, C, K, C == 2, ODD> : block_norm_queue_kernel<T, C, K, false, ODD>;
    // what a training step asks for, without branches around its parts (16384 x
    // 8192: 212 us instead of 225; 8192 x 4096 the same)
    if (keep && !ODD && p.c.post_norm && p.block_ckpt.codes && p.stream_ckpt.codes && p.normed && !p.block_out)
        kernel = block_norm_queue_kernel<T, C, K, C == 2, ODD, C == 2 && !ODD>;
    NormParams q = p;
    q.step_part = grid.x * p.ld_part;
    q.step_x = grid.x * p.ld_x;
    using Q = Queue<T, C, K, ODD>;
    const cudaError_t e = cudaFuncSetAttribute((const void*)kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               (int)Q::bytes(C == 2 ? 512 : 1024));
    if (e != cudaSuccess) return e;
    return launch_kernel(kernel, grid, threads, Q::bytes(threads), s, q);
}

template <class T>
cudaError_t launch(const NormParams& p, cudaStream_t s)
{
    constexpr int kItems = 12 / ((int)sizeof(T) / 2);        // 192 KiB of queues on an SM
    const int64_t groups = (p.c.cols + 255) / 256;
    if (p.c.cols <= 8192) {
        if (p.c.access == kAligned) return launch_queue<T, 2, kItems, false>(p, s);
        if (p.c.access == kOddPitch) return launch_queue<T, 2, kItems, true>(p, s);
    } else if (p.c.access == kAligned) {
        return launch_queue<T, 4, kItems / 4, false>(p, s);
    }
    const dim3 grid((unsigned)(p.c.rows < INT32_MAX ? p.c.rows : INT32_MAX));
    if (groups <= 32) return launch_kernel(block_norm_kernel<T, 2>, grid, (unsigned)((groups + 1) / 2) * 32, 0, s, p);
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
