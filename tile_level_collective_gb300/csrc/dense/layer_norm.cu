// Layer norm of a sum of N windows and a residual, in one pass over the rows.
//
// Bound by HBM: N + 1 reads and 2 writes per element with a residual. A block
// holds a row in registers (C chunks of 8 columns per thread), so that each
// element is read once although the mean and the deviations come before its last
// use; one wave of blocks walks the rows, and every warp keeps a queue of copies
// of its own columns of this row and the next ones in shared memory. Up to 8,192
// columns; wider rows take four chunks per thread.
//
// Measured on GB300 (bf16, of 6.8 TB/s copied): 8192 x 4096 with a residual 46 us
// (5.8 TB/s; straight from memory 57), 16384 x 8192 163 us (6.6 TB/s), of 8 parts
// 441 us (6.7 TB/s); without a residual 31 and 112 us (4.7 TB/s: latency at 16
// warps per SM, which issue in 61 % of the slots); 8192 x 4095 66 us; 4096 x 16384
// 100 us. One row of 7168 columns of 8 parts: 4.6 us in a graph.
#include "layers/layers_common.cuh"
#include "dense/dense_internal.h"
#include "host/host_checks.h"
#include "dense/row_stats.cuh"

namespace ptoc {

namespace {

// The bias' columns; zeros where there is none.
template <class T, int G>
__device__ __forceinline__ F8 load_bias8(const LayerNormParams& p, int32_t col, uint32_t mask)
{
    if (!p.bias) return F8{};
    return load_param8<T, G>(p.bias, p.param_f32, col, mask);
}

// What follows the sums s of the parts and the residual, for R rows in registers:
// `row` and those `step` rows apart, of which `rows` are there. KEEP: weight and
// bias are in w and b for all rows; else they are loaded for each row.
template <class T, int G, int C, int R, bool KEEP>
__device__ __forceinline__ void finish_rows(const LayerNormParams& p, int64_t row, int64_t step, int rows,
                                            F8 (&s)[R][C], const int32_t (&col)[C], const uint32_t (&mask)[C],
                                            const F8 (&w)[KEEP ? C : 1], const F8 (&b)[KEEP ? C : 1],
                                            RowStats<C, R>& stats)
{
    if (p.out)
#pragma unroll
        for (int r = 0; r < R; ++r)
            if (r < rows)
#pragma unroll
                for (int i = 0; i < C; ++i)
                    store8<T, G>((T*)p.out + (row + r * step) * p.ld_out, col[i], mask[i], s[r][i]);
    float mean[R], m2[R];
    stats.template of_rows<G>(s, mask, mean, m2);
#pragma unroll
    for (int r = 0; r < R; ++r) {
        if (r >= rows) break;
        const int64_t at = row + r * step;
        const float rstd = 1.0f / sqrtf(m2[r] * p.inv_cols + p.eps);
        if (p.stats && threadIdx.x == 0) {
            p.stats[at] = mean[r];
            p.stats[p.rows + at] = rstd;
        }
        const Pair shift = both(-mean[r]), scale = both(rstd);
#pragma unroll
        for (int i = 0; i < C; ++i) {
            F8 wi, bi;
            if constexpr (KEEP) {
                wi = w[i], bi = b[i];
            } else {
                wi = load_param8<T, G>(p.weight, p.param_f32, col[i], mask[i]);
                bi = load_bias8<T, G>(p, col[i], mask[i]);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j)
                s[r][i].p[j] = fma2(mul2(add2(s[r][i].p[j], shift), scale), wi.p[j], bi.p[j]);
            store8<T, G>((T*)p.normed + at * p.ld_normed, col[i], mask[i], s[r][i]);
        }
    }
}

// Through the warps' queues of K items: the parts and the residual of this row
// and of the next ones. KEEP: weight and bias stay in registers. R rows at a time
// share the exchanges between lanes and warps.
template <class T, int C, int K, bool ODD, int R>
__global__ void __launch_bounds__(C == 2 ? 512 : 1024, 1) layer_norm_queue_kernel(const LayerNormParams p)
{
    constexpr int G = ODD ? 1 : kVector<T>;
    constexpr bool KEEP = C == 2;
    pdl_enter();
    extern __shared__ __align__(16) unsigned char smem[];
    __shared__ __align__(16) float2 slots[RowStats<C, R>::kSlots];
    RowStats<C, R> stats(slots, p.cols);
    int32_t col[C];
    uint32_t mask[C];
    F8 w[KEEP ? C : 1], b[KEEP ? C : 1];
#pragma unroll
    for (int i = 0; i < C; ++i) {
        col[i] = first_col<G, C>(i);
        mask[i] = runs_below<G>(col[i], p.cols);
    }
    Queue<T, C, K, ODD> queue(smem, mask);
    // the item to copy next: source `src` (nparts: the residual) of row `ahead`
    const int items = p.nparts + (p.x != nullptr);
    int64_t ahead = blockIdx.x, part_at = ahead * p.ld_part;
    const T* x_row = (const T*)p.x + ahead * p.ld_x;
    int src = 0;
    auto push = [&] {
        queue.done();
        if (ahead < p.rows) {
            queue.copy_row(src < p.nparts ? (const T*)p.part[src] + part_at : x_row, col, mask, p.cols);
            if (++src == items) {
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
            w[i] = load_param8<T, G>(p.weight, p.param_f32, col[i], mask[i]);
            b[i] = load_bias8<T, G>(p, col[i], mask[i]);
        }
    for (int64_t row = blockIdx.x; row < p.rows; row += R * (int64_t)gridDim.x) {
        F8 s[R][C];
        const int rows = row + gridDim.x < p.rows ? R : 1;
#pragma unroll
        for (int k = 0; k < R; ++k) {
            if (k >= rows) {
#pragma unroll
                for (int i = 0; i < C; ++i) s[k][i] = F8{};
                break;
            }
            // where the rows begin in their words
            const uint32_t at = (uint32_t)(row + k * gridDim.x) * (uint32_t)sizeof(T);
            const uint32_t part_shift = at * (uint32_t)p.ld_part & 15u, x_shift = at * (uint32_t)p.ld_x & 15u;
            queue.wait();
#pragma unroll
            for (int i = 0; i < C; ++i) s[k][i] = queue.chunk(i, part_shift).expand();
            push();
            for (int r = 1; r < items; ++r) {
                const uint32_t shift = r < p.nparts ? part_shift : x_shift;
                queue.wait();
#pragma unroll
                for (int i = 0; i < C; ++i) {
                    const F8 f = queue.chunk(i, shift).expand();
#pragma unroll
                    for (int j = 0; j < 4; ++j) s[k][i].p[j] = add2(s[k][i].p[j], f.p[j]);
                }
                push();
            }
        }
        finish_rows<T, G, C, R, KEEP>(p, row, gridDim.x, rows, s, col, mask, w, b, stats);
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
}

// Rows straight from memory.
template <class T, int G, int C>
__global__ void __launch_bounds__(C == 2 ? 512 : 1024) layer_norm_kernel(const LayerNormParams p)
{
    pdl_enter();
    __shared__ __align__(16) float2 slots[RowStats<C, 1>::kSlots];
    RowStats<C, 1> stats(slots, p.cols);
    int32_t col[C];
    uint32_t mask[C];
#pragma unroll
    for (int i = 0; i < C; ++i) {
        col[i] = first_col<G, C>(i);
        mask[i] = runs_below<G>(col[i], p.cols);
    }
    for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
        F8 a[1][C];
        auto add = [&](const void* m, int64_t ld, bool first) {
#pragma unroll
            for (int i = 0; i < C; ++i) {
                const F8 f = load8<T, G>((const T*)m + row * ld, col[i], mask[i]).expand();
#pragma unroll
                for (int j = 0; j < 4; ++j) a[0][i].p[j] = first ? f.p[j] : add2(a[0][i].p[j], f.p[j]);
            }
        };
        add(p.part[0], p.ld_part, true);
        for (int r = 1; r < p.nparts; ++r) add(p.part[r], p.ld_part, false);
        if (p.x) add(p.x, p.ld_x, false);
        const F8 none[1] = {};
        finish_rows<T, G, C, 1, false>(p, row, 0, 1, a, col, mask, none, none, stats);
    }
}

template <class T, int G>
cudaError_t launch_direct(const LayerNormParams& p, cudaStream_t s)
{
    const int64_t groups = (p.cols + 255) / 256;             // warps' worth of chunks
    const dim3 grid((unsigned)(p.rows < INT32_MAX ? p.rows : INT32_MAX));
    if (groups <= 32)
        return launch_kernel(layer_norm_kernel<T, G, 2>, grid, (unsigned)((groups + 1) / 2) * 32, 0, s, p);
    return launch_kernel(layer_norm_kernel<T, G, 4>, grid, (unsigned)((groups + 3) / 4) * 32, 0, s, p);
}

template <class T, int C, int K, bool ODD, int R>
cudaError_t launch_rows(const LayerNormParams& p, cudaStream_t s)
{
    const int64_t groups = (p.cols + 255) / 256;
    const unsigned threads = (unsigned)((groups + C - 1) / C) * 32;
    // one wave: the registers and the queues of 512 threads of two chunks fill an SM
    const int64_t per_sm = C == 2 ? (512 / threads < 16 ? 512 / threads : 16) : 1;
    const int64_t most = 152 * per_sm;
    const dim3 grid((unsigned)(p.rows < most ? p.rows : most));
    using Q = Queue<T, C, K, ODD>;
    auto kernel = layer_norm_queue_kernel<T, C, K, ODD, R>;
    static std::atomic<uint64_t> done{0};
    LayerNormParams q = p;
    q.step_part = grid.x * p.ld_part;
    q.step_x = grid.x * p.ld_x;
    return launch_shared((const void*)kernel, (int)Q::bytes(C == 2 ? 512 : 1024), done,
                         [&] { return launch_kernel(kernel, grid, threads, Q::bytes(threads), s, q); });
}

// A row of one source is a short wait for memory and two exchanges, so two of
// them go together (16384 x 8192 bf16: 113 us instead of 135); of more sources
// they cost more than they give (with a residual 176 us instead of 167, 8192 x
// 4096 49 instead of 47: the copies come in longer bursts).
template <class T, int C, int K, bool ODD>
cudaError_t launch_queue(const LayerNormParams& p, cudaStream_t s)
{
    if (C == 2 && p.nparts == 1 && !p.x) return launch_rows<T, C, K, ODD, C == 2 ? 2 : 1>(p, s);
    return launch_rows<T, C, K, ODD, 1>(p, s);
}

template <class T>
cudaError_t launch(const LayerNormParams& p, cudaStream_t s)
{
    constexpr int kItems = 12 / ((int)sizeof(T) / 2);        // 192 KiB of queues on an SM
    if (p.cols <= 8192) {
        if (p.access == kAligned) return launch_queue<T, 2, kItems, false>(p, s);
        if (p.access == kOddPitch) return launch_queue<T, 2, kItems, true>(p, s);
    } else if (p.access == kAligned) {
        return launch_queue<T, 4, kItems / 4, false>(p, s);
    }
    return launch_direct<T, 1>(p, s);
}

}  // namespace

cudaError_t launch_layer_norm(const LayerNormParams& p, int dtype, cudaStream_t s)
{
    switch (dtype) {
    case PTOC_F32: return launch<float>(p, s);
    case PTOC_F16: return launch<__half>(p, s);
    default: return launch<__nv_bfloat16>(p, s);
    }
}

}  // namespace ptoc
