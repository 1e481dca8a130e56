// The backward pass of the norms around a block.
//
// With st = s * r, ah = a * ra, and gw the columns' factor (the weight of the
// norm after the block, times branch_scale and the gate where that varies
// along the columns; F is the rest, one number for the row):
//   ds = du + r * (wpre * dy - st * mean(wpre * dy * st));  d_residual = residual_scale * ds
//   t = gw * ds;  d_block = ra * F * (t - ah * mean(t * ah))
// The weights' and the gate's gradients need two sums over the rows for each
// column: of dy * st, and Q of ds * ah (times the gate where it varies by
// row), from which d_post_weight and the gate's gradient follow.
//
// Bound by HBM: per element it reads dy, du, s and a (the last two in 2 or 4
// bytes, or 33/32 as 8-bit checkpoints) and writes d_residual and d_block.
// One wave of blocks walks the rows with the two column sums in registers;
// copies of the next rows are queued in shared memory by each thread for
// itself, as in the forward pass. Each block writes its column sums as one
// partial row, and a second launch adds the partial rows in order.
#include "layers/layers_common.cuh"
#include "layers/layers_internal.h"

namespace ptoc {

namespace {

template <class T>
__device__ __forceinline__ float gate_of_row(const NormCommon& k, int64_t row)
{
    if (!k.gate) return 1.0f;
    return k.param_f32 ? ((const float*)k.gate)[row * k.gate_rs] : to_f32(((const T*)k.gate)[row * k.gate_rs]);
}

template <class T, int G>
__device__ __forceinline__ F8 gate8(const NormCommon& k, int64_t row, uint32_t col, uint32_t mask)
{
    return load_param8<T, G>((const char*)k.gate + row * k.gate_rs * (k.param_f32 ? 4 : (int)sizeof(T)), k.param_f32,
                             col, mask);
}

// Where the per-column parameters of chunk i come from: f32 copies that the
// thread keeps in shared memory (KEEP), or memory.
template <class T, int G, int C, bool KEEP>
struct Columns {
    const NormCommon& k;
    const uint32_t (&col)[C];
    const uint32_t (&mask)[C];
    uint32_t kept;                          // [2][C][2][threads] 16-byte words: wpre, then the factor

    __device__ __forceinline__ F8 pre(int i) const
    {
        if constexpr (KEEP) return read(2 * i);
        return load_param8<T, G>(k.pre_weight, k.param_f32, col[i], mask[i]);
    }
    // the weight of the norm after the block, times branch_scale * gate for a gate of columns
    __device__ __forceinline__ F8 factor(int i) const
    {
        if constexpr (KEEP) return read(2 * (C + i));
        return load_factor(i);
    }
    __device__ __forceinline__ F8 load_factor(int i) const
    {
        F8 w = load_param8<T, G>(k.post_weight, k.param_f32, col[i], mask[i]);
        if (k.gate_cs && !k.gate_rs) {
            const F8 g = gate8<T, G>(k, 0, col[i], mask[i]);
#pragma unroll
            for (int j = 0; j < 4; ++j) w.p[j] = mul2(w.p[j], mul2(both(k.branch_scale), g.p[j]));
        }
        return w;
    }
    __device__ __forceinline__ uint32_t word(int n) const { return kept + (uint32_t)(n * 16) * blockDim.x; }
    __device__ __forceinline__ F8 read(int n) const
    {
        F8 f;
#pragma unroll
        for (int h = 0; h < 2; ++h)
            asm volatile("ld.shared.v2.u64 {%0, %1}, [%2];" : "=l"(f.p[2 * h]), "=l"(f.p[2 * h + 1]) : "r"(word(n + h))
                         : "memory");
        return f;
    }
    __device__ __forceinline__ void keep(int n, const F8& f) const
    {
#pragma unroll
        for (int h = 0; h < 2; ++h)
            asm volatile("st.shared.v2.u64 [%0], {%1, %2};" ::"r"(word(n + h)), "l"(f.p[2 * h]), "l"(f.p[2 * h + 1])
                         : "memory");
    }
};

// One row. The loader gives, chunk by chunk and in this order: the stream
// times a factor, dy, du (if p.du), the block output times a factor.
template <class T, int G, int C, bool KEEP, class Loader>
__device__ __forceinline__ void back_row(const NormBackParams& p, int64_t row, Loader& in,
                                         const Columns<T, G, C, KEEP>& cols, F8 (&sum_pre)[C], F8 (&sum_q)[C],
                                         float& sum_scalar, float (*slots)[32], int& turn)
{
    const NormCommon& k = p.c;
    const uint32_t (&col)[C] = cols.col;
    const uint32_t (&mask)[C] = cols.mask;
    const float ra = k.post_norm ? p.rstd[row] : 1.0f, r = p.rstd[k.rows + row];
    const bool by_column = k.gate_cs != 0, by_element = by_column && k.gate_rs != 0;
    const float g_row = by_column ? 1.0f : gate_of_row<T>(k, row);
    F8 st[C], up[C];
    Pair dot = 0;
    in.begin_stream();
#pragma unroll
    for (int i = 0; i < C; ++i) st[i] = in.stream(i, r);
    in.end();
    in.begin_matrix(p.dy, p.ld_dy);
#pragma unroll
    for (int i = 0; i < C; ++i) {
        const F8 dy = in.matrix(i).expand(), w = cols.pre(i);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            up[i].p[j] = mul2(w.p[j], dy.p[j]);
            sum_pre[i].p[j] = fma2(dy.p[j], st[i].p[j], sum_pre[i].p[j]);
            dot = fma2(up[i].p[j], st[i].p[j], dot);
        }
    }
    in.end();
    float total[1] = {sum_of(dot)};
    block_sum(total, slots[turn]);
    turn ^= 1;
    // up becomes ds
    const Pair m = both(-total[0] * k.inv_cols), r2 = both(r);
    if (p.du) {
        in.begin_matrix(p.du, p.ld_du);
#pragma unroll
        for (int i = 0; i < C; ++i) {
            const F8 du = in.matrix(i).expand();
#pragma unroll
            for (int j = 0; j < 4; ++j) up[i].p[j] = fma2(r2, fma2(m, st[i].p[j], up[i].p[j]), du.p[j]);
        }
        in.end();
    } else {
#pragma unroll
        for (int i = 0; i < C; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) up[i].p[j] = mul2(r2, fma2(m, st[i].p[j], up[i].p[j]));
    }
    // st becomes ah
    in.begin_block();
#pragma unroll
    for (int i = 0; i < C; ++i) st[i] = in.block(i, ra);
    in.end();
    const bool q_scaled = !by_column && k.gate_rs;       // a gate that varies by row goes into Q
    dot = 0;
#pragma unroll
    for (int i = 0; i < C; ++i) {
        F8 w;
#pragma unroll
        for (int j = 0; j < 4; ++j) w.p[j] = mul2(both(k.residual_scale), up[i].p[j]);
        store8<T, G>((T*)p.d_residual + row * p.ld_dres, col[i], mask[i], w);
        w = cols.factor(i);
        if (by_element) {
            const F8 g = gate8<T, G>(k, row, col[i], mask[i]);
            if (p.gate_kind == kGateElement) {
                F8 d;
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    d.p[j] = mul2(both(k.branch_scale), mul2(up[i].p[j], mul2(st[i].p[j], w.p[j])));
                // packed rows of floats, whose alignment follows the number of columns
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    float v[2];
                    split(d.p[j / 2], v[0], v[1]);
                    if (mask[i] >> (j / G) & 1) p.d_gate[row * k.cols + col[i] + j / G * 32 * G + j % G] = v[j & 1];
                }
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                sum_q[i].p[j] = fma2(mul2(g.p[j], up[i].p[j]), st[i].p[j], sum_q[i].p[j]);
                w.p[j] = mul2(w.p[j], mul2(both(k.branch_scale), g.p[j]));
            }
        } else if (q_scaled) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                sum_q[i].p[j] = fma2(mul2(both(g_row), up[i].p[j]), st[i].p[j], sum_q[i].p[j]);
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) sum_q[i].p[j] = fma2(up[i].p[j], st[i].p[j], sum_q[i].p[j]);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            up[i].p[j] = mul2(up[i].p[j], w.p[j]);
            dot = fma2(up[i].p[j], st[i].p[j], dot);
        }
    }
    total[0] = sum_of(dot);
    const bool row_gate = p.gate_kind == kGateToken || p.gate_kind == kGateScalar;
    if (k.post_norm || row_gate) {
        block_sum(total, slots[turn]);
        turn ^= 1;
    }
    if (row_gate) {
        const float d = k.branch_scale * total[0];
        if (p.gate_kind == kGateToken && threadIdx.x == 0) p.d_gate[row] = d;
        sum_scalar += d;
    }
    const Pair m2 = both(k.post_norm ? -total[0] * k.inv_cols : 0.0f);
    const Pair f = both(ra * (by_column ? 1.0f : k.branch_scale * g_row));
#pragma unroll
    for (int i = 0; i < C; ++i) {
#pragma unroll
        for (int j = 0; j < 4; ++j) up[i].p[j] = mul2(f, fma2(m2, st[i].p[j], up[i].p[j]));
        store8<T, G>((T*)p.d_block + row * p.ld_dblk, col[i], mask[i], up[i]);
    }
}

// This block's partial rows of the column sums.
template <int G, int C>
__device__ __forceinline__ void store_sums(const NormBackParams& p, const uint32_t (&col)[C], const uint32_t (&mask)[C],
                                           const F8 (&sum_pre)[C], const F8 (&sum_q)[C], float sum_scalar)
{
    const int64_t cols = p.c.cols, plane = (int64_t)gridDim.x * cols;
    float* mine = p.partial + (int64_t)blockIdx.x * cols;
#pragma unroll
    for (int i = 0; i < C; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            float a[2], b[2];
            split(sum_pre[i].p[j / 2], a[0], a[1]);
            split(sum_q[i].p[j / 2], b[0], b[1]);
            if (mask[i] >> (j / G) & 1) {
                float* at = mine + col[i] + j / G * 32 * G + j % G;
                if (p.d_pre) at[0] = a[j & 1];
                if (p.need_q) at[plane] = b[j & 1];
            }
        }
    if (p.gate_kind == kGateScalar && threadIdx.x == 0) p.partial[2 * plane + blockIdx.x] = sum_scalar;
}

// Chunks from the thread's queue, in the order of the items: stream, dy, du, block.
template <class T, int C, int K>
struct QueueLoader {
    static constexpr int G = kVector<T>;
    const NormBackParams& p;
    Queue<T, C, K> queue;
    const uint32_t (&col)[C];
    const uint32_t (&mask)[C];
    int64_t ahead;                          // the row of the item to copy next
    int item;
    static constexpr int kRuns = 8 / G;
    uint32_t s_exp[C * kRuns], a_exp[C * kRuns], s_next[C * kRuns], a_next[C * kRuns];   // exponent bytes of this row and the next

    __device__ __forceinline__ QueueLoader(const NormBackParams& q, void* smem, const uint32_t (&c)[C],
                                           const uint32_t (&m)[C])
        : p(q), queue(smem), col(c), mask(m), ahead(blockIdx.x), item(0)
    {
#pragma unroll 1
        for (int k = 0; k < K; ++k) push();
        exponents(blockIdx.x);
    }
    __device__ __forceinline__ void push()
    {
        if (ahead < p.c.rows) {
            if (item == 0) {
                if (p.stream) queue.copy_row((const T*)p.stream + ahead * p.ld_stream, col, mask);
                else queue.copy_codes(p.stream_ckpt.codes + ahead * p.stream_ckpt.ld_codes, col, mask);
            } else if (item == 1) {
                queue.copy_row((const T*)p.dy + ahead * p.ld_dy, col, mask);
            } else if (item == 2) {
                queue.copy_row((const T*)p.du + ahead * p.ld_du, col, mask);
            } else {
                if (p.block) queue.copy_row((const T*)p.block + ahead * p.ld_block, col, mask);
                else queue.copy_codes(p.block_ckpt.codes + ahead * p.block_ckpt.ld_codes, col, mask);
            }
            item += item == 1 && !p.du ? 2 : 1;
            if (item == 4) item = 0, ahead += gridDim.x;
        }
        queue.next();
    }
    // Read a row's exponent bytes, a row before their use.
    __device__ __forceinline__ void exponents(int64_t row)
    {
        const bool in = row < p.c.rows;
        const uint8_t* s = p.stream ? nullptr : p.stream_ckpt.exps + row * p.stream_ckpt.ld_exps;
        const uint8_t* a = p.block ? nullptr : p.block_ckpt.exps + row * p.block_ckpt.ld_exps;
#pragma unroll
        for (int i = 0; i < C; ++i)
#pragma unroll
            for (int q = 0; q < kRuns; ++q) {
                const bool on = in && (mask[i] >> q & 1);
                const uint32_t b = (col[i] + q * 32 * G) >> 5;
                s_next[i * kRuns + q] = s && on ? s[b] : 0u;
                a_next[i * kRuns + q] = a && on ? a[b] : 0u;
            }
    }
    __device__ __forceinline__ void row(int64_t r)
    {
#pragma unroll
        for (int i = 0; i < C * kRuns; ++i) s_exp[i] = s_next[i], a_exp[i] = a_next[i];
        exponents(r + gridDim.x);
    }
    __device__ __forceinline__ void begin_stream() { queue.wait(); }
    __device__ __forceinline__ void begin_block() { queue.wait(); }
    __device__ __forceinline__ void begin_matrix(const void*, int64_t) { queue.wait(); }
    __device__ __forceinline__ void end() { push(); }
    __device__ __forceinline__ Raw8<T, G> matrix(int i) const { return queue.chunk(i); }
    __device__ __forceinline__ F8 saved(int i, bool whole, const uint32_t* bytes, float factor) const
    {
        if (whole) {
            F8 f = queue.chunk(i).expand();
#pragma unroll
            for (int j = 0; j < 4; ++j) f.p[j] = mul2(f.p[j], both(factor));
            return f;
        }
        CkptRaw<G> k;
        queue.codes(i, k.w);
#pragma unroll
        for (int q = 0; q < kRuns; ++q) k.byte[q] = bytes[i * kRuns + q];
        return ckpt_values<G>(k, factor);
    }
    __device__ __forceinline__ F8 stream(int i, float f) const { return saved(i, p.stream, s_exp, f); }
    __device__ __forceinline__ F8 block(int i, float f) const { return saved(i, p.block, a_exp, f); }
};

constexpr int kQueueThreads = 512;

template <class T, int K>
__global__ void __launch_bounds__(kQueueThreads) norm_backward_queue_kernel(const NormBackParams p)
{
    constexpr int C = 2, G = kVector<T>;
    pdl_enter();
    extern __shared__ __align__(16) unsigned char smem[];
    __shared__ float slots[2][32];
    int turn = 0;                           // block_sum's slots in turn
    uint32_t col[C], mask[C];
#pragma unroll
    for (int i = 0; i < C; ++i) {
        col[i] = first_col<G>(i);
        mask[i] = runs_below<G>(col[i], p.c.cols);
    }
    QueueLoader<T, C, K> in(p, smem + (size_t)blockDim.x * C * 2 * 32, col, mask);
    const Columns<T, G, C, true> cols{p.c, col, mask, (uint32_t)__cvta_generic_to_shared(smem) + threadIdx.x * 16};
    const Columns<T, G, C, false> memory{p.c, col, mask, 0};
#pragma unroll
    for (int i = 0; i < C; ++i) {
        cols.keep(2 * i, memory.pre(i));
        cols.keep(2 * (C + i), memory.load_factor(i));
    }
    F8 sum_pre[C] = {}, sum_q[C] = {};
    float sum_scalar = 0.0f;
    for (int64_t row = blockIdx.x; row < p.c.rows; row += gridDim.x) {
        in.row(row);
        back_row<T, G, C, true>(p, row, in, cols, sum_pre, sum_q, sum_scalar, slots, turn);
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    store_sums<G, C>(p, col, mask, sum_pre, sum_q, sum_scalar);
}

// Chunks straight from memory, for rows at any address and very wide ones.
template <class T, int G, int C>
struct DirectLoader {
    const NormBackParams& p;
    const uint32_t (&col)[C];
    const uint32_t (&mask)[C];
    int64_t row;
    CkptRaw<G> codes[C];
    Raw8<T, G> whole[C];

    __device__ __forceinline__ void end() {}
    __device__ __forceinline__ void fetch(const void* m, int64_t ld, const ptoc_ckpt8& k)
    {
        const Ckpt c{k.codes, k.exps, k.ld_codes, k.ld_exps};
        if (m) begin_matrix(m, ld);
        else
#pragma unroll
            for (int i = 0; i < C; ++i) codes[i] = ckpt_load8<G>(c, row, col[i], mask[i]);
    }
    __device__ __forceinline__ void begin_stream() { fetch(p.stream, p.ld_stream, p.stream_ckpt); }
    __device__ __forceinline__ void begin_block() { fetch(p.block, p.ld_block, p.block_ckpt); }
    __device__ __forceinline__ void begin_matrix(const void* m, int64_t ld)
    {
#pragma unroll
        for (int i = 0; i < C; ++i) whole[i] = load8<T, G>((const T*)m + row * ld, col[i], mask[i]);
    }
    __device__ __forceinline__ const Raw8<T, G>& matrix(int i) const { return whole[i]; }
    __device__ __forceinline__ F8 saved(int i, bool matrix, float factor) const
    {
        if (!matrix) return ckpt_values<G>(codes[i], factor);
        F8 f = whole[i].expand();
#pragma unroll
        for (int j = 0; j < 4; ++j) f.p[j] = mul2(f.p[j], both(factor));
        return f;
    }
    __device__ __forceinline__ F8 stream(int i, float f) const { return saved(i, p.stream, f); }
    __device__ __forceinline__ F8 block(int i, float f) const { return saved(i, p.block, f); }
};

template <class T, int G, int C>
__global__ void __launch_bounds__(C == 2 ? 512 : 1024) norm_backward_kernel(const NormBackParams p)
{
    pdl_enter();
    __shared__ float slots[2][32];
    int turn = 0;
    uint32_t col[C], mask[C];
#pragma unroll
    for (int i = 0; i < C; ++i) {
        col[i] = first_col<G>(i);
        mask[i] = runs_below<G>(col[i], p.c.cols);
    }
    const Columns<T, G, C, false> cols{p.c, col, mask, 0};
    F8 sum_pre[C] = {}, sum_q[C] = {};
    float sum_scalar = 0.0f;
    for (int64_t row = blockIdx.x; row < p.c.rows; row += gridDim.x) {
        DirectLoader<T, G, C> in{p, col, mask, row};
        back_row<T, G, C, false>(p, row, in, cols, sum_pre, sum_q, sum_scalar, slots, turn);
    }
    store_sums<G, C>(p, col, mask, sum_pre, sum_q, sum_scalar);
}

// Sums of the partial rows: a block takes 32 columns of one kind; its 8 warps
// each add a run of the partial rows in order, and the runs are added in
// order. Kind 0: d_pre; 1: Q, from which d_post and the gradient of a gate of
// columns follow; 2: the gradient of a scalar gate.
template <class T>
__global__ void __launch_bounds__(kBlock) norm_backward_sum_kernel(const NormBackParams p)
{
    pdl_enter();
    __shared__ float runs[kBlock / 32][32];
    const NormCommon& k = p.c;
    const int64_t plane = (int64_t)p.grid * k.cols;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t col = (int64_t)blockIdx.x * 32 + lane;
    const int kind = blockIdx.y;
    const bool live = kind == 0 ? p.d_pre && col < k.cols
                    : kind == 1 ? p.need_q && col < k.cols
                                : p.gate_kind == kGateScalar && col == 0;
    float sum = 0.0f;
    if (live) {
        const float* src = p.partial + kind * plane + col;
        const int64_t step = kind == 2 ? 1 : k.cols;
        const int per = (p.grid + kBlock / 32 - 1) / (kBlock / 32);
        const int end = min(p.grid, (warp + 1) * per);
#pragma unroll 8
        for (int b = warp * per; b < end; ++b) sum += src[b * step];
    }
    runs[warp][lane] = sum;
    __syncthreads();
    if (warp || !live) return;
    sum = 0.0f;
#pragma unroll
    for (int w = 0; w < kBlock / 32; ++w) sum += runs[w][lane];
    auto param = [&](const void* q, int64_t i) {
        return !q ? 1.0f : k.param_f32 ? ((const float*)q)[i] : to_f32(((const T*)q)[i]);
    };
    if (kind == 0) {
        p.d_pre[col] = sum;
    } else if (kind == 2) {
        p.d_gate[0] = sum;
    } else {
        // a gate that varies by row is in Q already
        if (p.d_post) p.d_post[col] = k.branch_scale * (k.gate_rs ? sum : param(k.gate, k.gate_cs ? col : 0) * sum);
        if (p.gate_kind == kGateChannel) p.d_gate[col] = k.branch_scale * (param(k.post_weight, col) * sum);
    }
}

// The queue form: items in flight and its rule. Two chunks per thread and 512
// threads on an SM; wider rows leave no room for two rows of copies.
template <class T>
constexpr int kItems = 8 / ((int)sizeof(T) / 2);
constexpr int64_t kQueueCols = kQueueThreads * 16;

template <class T>
cudaError_t launch(const NormBackParams& p, cudaStream_t s)
{
    const dim3 grid((unsigned)p.grid);
    const int64_t groups = (p.c.cols + 255) / 256;
    cudaError_t e;
    if (p.c.vec && p.c.cols <= kQueueCols) {
        const unsigned threads = (unsigned)((groups + 1) / 2) * 32;
        const size_t per_thread = 2 * (2 * 32 + (size_t)kItems<T> * sizeof(T) * 8);
        auto kernel = norm_backward_queue_kernel<T, kItems<T>>;
        e = cudaFuncSetAttribute((const void*)kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 (int)(per_thread * kQueueThreads));
        if (e == cudaSuccess) e = launch_kernel(kernel, grid, threads, per_thread * threads, s, p);
    } else if (p.c.vec) {
        e = launch_kernel(norm_backward_kernel<T, kVector<T>, 4>, grid, (unsigned)((groups + 3) / 4) * 32, 0, s, p);
    } else if (p.c.cols <= kQueueCols) {
        e = launch_kernel(norm_backward_kernel<T, 1, 2>, grid, (unsigned)((groups + 1) / 2) * 32, 0, s, p);
    } else {
        e = launch_kernel(norm_backward_kernel<T, 1, 4>, grid, (unsigned)((groups + 3) / 4) * 32, 0, s, p);
    }
    if (e != cudaSuccess) return e;
    if (!p.d_pre && !p.need_q && p.gate_kind != kGateScalar) return cudaSuccess;
    const dim3 sums((unsigned)((p.c.cols + 31) / 32), p.gate_kind == kGateScalar ? 3 : 2);
    return launch_kernel(norm_backward_sum_kernel<T>, sums, kBlock, 0, s, p);
}

}  // namespace

// One wave: the blocks that 512 threads of two chunks on each SM make up. The
// count is GB300's, not the device's answer: the order of the sums and the
// workspace then depend on the sizes alone.
int norm_backward_grid(int64_t rows, int64_t cols)
{
    constexpr int kSms = 152;
    const int64_t threads = (cols + 511) / 512 * 32;
    const int64_t per_sm = threads >= 512 ? 1 : 512 / threads < 16 ? 512 / threads : 16;
    const int64_t most = (int64_t)kSms * per_sm;
    return (int)(rows < most ? rows : most);
}

cudaError_t launch_block_norm_backward(const NormBackParams& p, int dtype, cudaStream_t s)
{
    switch (dtype) {
    case PTOC_F32: return launch<float>(p, s);
    case PTOC_F16: return launch<__half>(p, s);
    default: return launch<__nv_bfloat16>(p, s);
    }
}

}  // namespace ptoc
