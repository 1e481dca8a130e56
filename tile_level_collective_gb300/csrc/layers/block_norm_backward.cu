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

template <class T, bool V>
__device__ __forceinline__ void gate8(const NormCommon& k, int64_t row, int64_t c, uint32_t mask, float* g)
{
    load_param8<T, V>((const char*)k.gate + row * k.gate_rs * (k.param_f32 ? 4 : (int)sizeof(T)), k.param_f32, c, mask, g);
}

// Where the per-column parameters of chunk i come from: f32 copies that the
// thread keeps in shared memory (KEEP), or memory.
template <class T, bool V, bool KEEP>
struct Columns {
    const NormCommon& k;
    const float* kept;            // [2][C][2][threads] float4: wpre, then gw
    __device__ __forceinline__ void pre(int i, int64_t c, uint32_t mask, float* w) const
    {
        if constexpr (KEEP) read(2 * i, w);
        else load_param8<T, V>(k.pre_weight, k.param_f32, c, mask, w);
    }
    // the weight of the norm after the block, times branch_scale * gate for a gate of columns
    __device__ __forceinline__ void factor(int i, int C, int64_t c, uint32_t mask, float* w) const
    {
        if constexpr (KEEP) read(2 * (C + i), w);
        else load_factor(c, mask, w);
    }
    __device__ __forceinline__ void load_factor(int64_t c, uint32_t mask, float* w) const
    {
        load_param8<T, V>(k.post_weight, k.param_f32, c, mask, w);
        if (k.gate_cs && !k.gate_rs) {
            float g[8];
            gate8<T, V>(k, 0, c, mask, g);
#pragma unroll
            for (int j = 0; j < 8; ++j) w[j] *= k.branch_scale * g[j];
        }
    }
    __device__ __forceinline__ void read(int slot, float* w) const
    {
        const float4* p = (const float4*)kept + (int64_t)slot * blockDim.x + threadIdx.x;
        const float4 a = p[0], b = p[blockDim.x];
        w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w, w[4] = b.x, w[5] = b.y, w[6] = b.z, w[7] = b.w;
    }
    static __device__ __forceinline__ void keep(float* kept, int slot, const float* w)
    {
        float4* p = (float4*)kept + (int64_t)slot * blockDim.x + threadIdx.x;
        p[0] = make_float4(w[0], w[1], w[2], w[3]);
        p[blockDim.x] = make_float4(w[4], w[5], w[6], w[7]);
    }
};

// One row. Loader gives, chunk by chunk and in this order: stream(i, factor),
// dy(i), du(i) (if p.du), block(i, factor).
template <class T, bool V, int C, bool KEEP, class Loader>
__device__ __forceinline__ void back_row(const NormBackParams& p, int64_t row, Loader& in, const uint32_t (&mask)[C],
                                         const Columns<T, V, KEEP>& cols, float (&sum_pre)[C][8], float (&sum_q)[C][8],
                                         float& sum_scalar, float (*slots)[32], int& turn)
{
    const NormCommon& k = p.c;
    const float ra = k.post_norm ? p.rstd[row] : 1.0f, r = p.rstd[k.rows + row];
    const bool by_column = k.gate_cs != 0, by_element = by_column && k.gate_rs != 0;
    const float g_row = by_column ? 1.0f : gate_of_row<T>(k, row);
    float st[C][8], up[C][8];
    float dot[1] = {0.0f};
    in.begin_stream();
#pragma unroll
    for (int i = 0; i < C; ++i) in.stream(i, r, st[i]);
    in.end();
    in.begin();
#pragma unroll
    for (int i = 0; i < C; ++i) {
        const Raw8<T> dy = in.matrix(i, p.dy, p.ld_dy);
        float w[8];
        cols.pre(i, (int64_t)i * blockDim.x + threadIdx.x, mask[i], w);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            up[i][j] = w[j] * dy.at(j);
            sum_pre[i][j] += dy.at(j) * st[i][j];
            dot[0] += up[i][j] * st[i][j];
        }
    }
    in.end();
    block_sum(dot, slots[turn]);
    turn ^= 1;
    const float m = dot[0] * k.inv_cols;
#pragma unroll
    for (int i = 0; i < C; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) up[i][j] = r * (up[i][j] - m * st[i][j]);
    if (p.du) {
        in.begin();
#pragma unroll
        for (int i = 0; i < C; ++i) {
            const Raw8<T> du = in.matrix(i, p.du, p.ld_du);
#pragma unroll
            for (int j = 0; j < 8; ++j) up[i][j] += du.at(j);
        }
        in.end();
    }
    // up holds ds; st becomes ah
    in.begin_block();
#pragma unroll
    for (int i = 0; i < C; ++i) in.block(i, ra, st[i]);
    in.end();
    const float q_row = by_column ? 1.0f : (k.gate_rs ? g_row : 1.0f);       // a gate that varies by row goes into Q
    float dots[1] = {0.0f};
#pragma unroll
    for (int i = 0; i < C; ++i) {
        const int64_t c = (int64_t)i * blockDim.x + threadIdx.x;
        float w[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) w[j] = k.residual_scale * up[i][j];
        store8<T, V>((T*)p.d_residual + row * p.ld_dres, c, mask[i], w);
        cols.factor(i, C, c, mask[i], w);
        if (by_element) {
            float g[8];
            gate8<T, V>(k, row, c, mask[i], g);
            if (p.gate_kind == kGateElement)
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (mask[i] >> j & 1)
                        p.d_gate[row * k.cols + col_of<V>(c, j)] = k.branch_scale * (up[i][j] * (st[i][j] * w[j]));
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                sum_q[i][j] += g[j] * up[i][j] * st[i][j];
                w[j] *= k.branch_scale * g[j];
            }
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) sum_q[i][j] += q_row * up[i][j] * st[i][j];
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            up[i][j] *= w[j];
            dots[0] += up[i][j] * st[i][j];
        }
    }
    const bool row_gate = p.gate_kind == kGateToken || p.gate_kind == kGateScalar;
    if (k.post_norm || row_gate) {
        block_sum(dots, slots[turn]);
        turn ^= 1;
    }
    if (row_gate) {
        const float d = k.branch_scale * dots[0];
        if (p.gate_kind == kGateToken && threadIdx.x == 0) p.d_gate[row] = d;
        sum_scalar += d;
    }
    const float m2 = k.post_norm ? dots[0] * k.inv_cols : 0.0f;
    const float f = ra * (by_column ? 1.0f : k.branch_scale * g_row);
#pragma unroll
    for (int i = 0; i < C; ++i) {
        float v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = f * (up[i][j] - m2 * st[i][j]);
        store8<T, V>((T*)p.d_block + row * p.ld_dblk, (int64_t)i * blockDim.x + threadIdx.x, mask[i], v);
    }
}

// This block's partial rows of the column sums.
template <bool V, int C>
__device__ __forceinline__ void store_sums(const NormBackParams& p, const uint32_t (&mask)[C],
                                           const float (&sum_pre)[C][8], const float (&sum_q)[C][8], float sum_scalar)
{
    const int64_t cols = p.c.cols, plane = (int64_t)gridDim.x * cols;
    float* mine = p.partial + (int64_t)blockIdx.x * cols;
#pragma unroll
    for (int i = 0; i < C; ++i) {
        const int64_t c = (int64_t)i * blockDim.x + threadIdx.x;
        if (p.d_pre) store8<float, V>(mine, c, mask[i], sum_pre[i]);
        if (p.need_q) store8<float, V>(mine + plane, c, mask[i], sum_q[i]);
    }
    if (p.gate_kind == kGateScalar && threadIdx.x == 0) p.partial[2 * plane + blockIdx.x] = sum_scalar;
}

// Chunks from the thread's queue, in the order of the items: stream, dy, du, block.
template <class T, int C, int K>
struct QueueLoader {
    const NormBackParams& p;
    Queue<C, (int)sizeof(T) / 2, K> queue;
    const uint32_t (&mask)[C];
    int64_t ahead;                          // the row of the item to copy next
    int item;
    uint32_t s_exp[C], a_exp[C], s_next[C], a_next[C];   // exponent bytes of this row and the next

    __device__ __forceinline__ QueueLoader(const NormBackParams& q, void* smem, const uint32_t (&m)[C])
        : p(q), queue(smem), mask(m), ahead(blockIdx.x), item(0)
    {
#pragma unroll
        for (int i = 0; i < C; ++i)
            if (!mask[i]) queue.clear(i);
#pragma unroll 1
        for (int k = 0; k < K; ++k) push();
        exponents(blockIdx.x);
    }
    __device__ __forceinline__ void codes(const ptoc_ckpt8& k)
    {
#pragma unroll
        for (int i = 0; i < C; ++i)
            queue.copy8(i, k.codes + ahead * k.ld_codes + ((int64_t)i * blockDim.x + threadIdx.x) * 8, mask[i] != 0);
    }
    __device__ __forceinline__ void push()
    {
        if (ahead < p.c.rows) {
            if (item == 0) {
                if (p.stream) queue.template copy_row<T>((const T*)p.stream + ahead * p.ld_stream, mask);
                else codes(p.stream_ckpt);
            } else if (item == 1) {
                queue.template copy_row<T>((const T*)p.dy + ahead * p.ld_dy, mask);
            } else if (item == 2) {
                queue.template copy_row<T>((const T*)p.du + ahead * p.ld_du, mask);
            } else {
                if (p.block) queue.template copy_row<T>((const T*)p.block + ahead * p.ld_block, mask);
                else codes(p.block_ckpt);
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
#pragma unroll
        for (int i = 0; i < C; ++i) {
            const int64_t b = ((int64_t)i * blockDim.x + threadIdx.x) >> 2;
            s_next[i] = a_next[i] = 0;
            if (!p.stream) s_next[i] = load1_if(p.stream_ckpt.exps + row * p.stream_ckpt.ld_exps + b, in && mask[i]);
            if (!p.block) a_next[i] = load1_if(p.block_ckpt.exps + row * p.block_ckpt.ld_exps + b, in && mask[i]);
        }
    }
    __device__ __forceinline__ void row(int64_t r)
    {
#pragma unroll
        for (int i = 0; i < C; ++i) s_exp[i] = s_next[i], a_exp[i] = a_next[i];
        exponents(r + gridDim.x);
    }
    __device__ __forceinline__ void begin() { queue.wait(); }
    __device__ __forceinline__ void begin_stream() { queue.wait(); }
    __device__ __forceinline__ void begin_block() { queue.wait(); }
    __device__ __forceinline__ void end() { push(); }
    __device__ __forceinline__ Raw8<T> matrix(int i, const void*, int64_t) const { return queue.template chunk<T>(i); }
    __device__ __forceinline__ void saved(int i, bool whole, uint32_t byte, float factor, float* v) const
    {
        if (whole) {
            const Raw8<T> w = queue.template chunk<T>(i);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = w.at(j) * factor;
        } else {
            const Words<4> w = queue.read(i, 0);
            CkptRaw<true> k;
            k.w[0] = w.w[0];
            k.w[1] = w.w[1];
            k.byte = byte;
            ckpt_values<true>(k, factor, v);
        }
    }
    __device__ __forceinline__ void stream(int i, float f, float* v) const { saved(i, p.stream, s_exp[i], f, v); }
    __device__ __forceinline__ void block(int i, float f, float* v) const { saved(i, p.block, a_exp[i], f, v); }
};

constexpr int kQueueThreads = 512;

template <class T, int K>
__global__ void __launch_bounds__(kQueueThreads) norm_backward_queue_kernel(const NormBackParams p)
{
    constexpr int C = 2;
    pdl_enter();
    extern __shared__ __align__(16) unsigned char smem[];
    __shared__ float slots[2][32];
    int turn = 0;                           // block_sum's slots in turn
    uint32_t mask[C];
#pragma unroll
    for (int i = 0; i < C; ++i) mask[i] = chunk_mask<true>((int64_t)i * blockDim.x + threadIdx.x, p.c.cols);
    float* kept = (float*)smem;
    QueueLoader<T, C, K> in(p, smem + (size_t)blockDim.x * C * 2 * 32, mask);
    const Columns<T, true, false> memory{p.c, nullptr};
    const Columns<T, true, true> cols{p.c, kept};
#pragma unroll
    for (int i = 0; i < C; ++i) {
        const int64_t c = (int64_t)i * blockDim.x + threadIdx.x;
        float w[8];
        memory.pre(i, c, mask[i], w);
        cols.keep(kept, 2 * i, w);
        memory.load_factor(c, mask[i], w);
        cols.keep(kept, 2 * (C + i), w);
    }
    float sum_pre[C][8] = {}, sum_q[C][8] = {};
    float sum_scalar = 0.0f;
    for (int64_t row = blockIdx.x; row < p.c.rows; row += gridDim.x) {
        in.row(row);
        back_row<T, true, C, true>(p, row, in, mask, cols, sum_pre, sum_q, sum_scalar, slots, turn);
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    store_sums<true, C>(p, mask, sum_pre, sum_q, sum_scalar);
}

// Chunks straight from memory, for rows at any address and very wide ones.
template <class T, bool V, int C>
struct DirectLoader {
    const NormBackParams& p;
    const uint32_t (&mask)[C];
    int64_t row;
    CkptRaw<V> codes[C];
    Raw8<T> whole[C];

    __device__ __forceinline__ int64_t chunk(int i) const { return (int64_t)i * blockDim.x + threadIdx.x; }
    __device__ __forceinline__ void begin() {}
    __device__ __forceinline__ void end() {}
    __device__ __forceinline__ void fetch(const void* m, int64_t ld, const ptoc_ckpt8& k)
    {
        const Ckpt c{k.codes, k.exps, k.ld_codes, k.ld_exps};
#pragma unroll
        for (int i = 0; i < C; ++i) {
            if (m) whole[i] = load8<T, V>((const T*)m + row * ld, chunk(i), mask[i]);
            else codes[i] = ckpt_load8<V>(c, row, chunk(i), mask[i]);
        }
    }
    __device__ __forceinline__ void begin_stream() { fetch(p.stream, p.ld_stream, p.stream_ckpt); }
    __device__ __forceinline__ void begin_block() { fetch(p.block, p.ld_block, p.block_ckpt); }
    __device__ __forceinline__ Raw8<T> matrix(int i, const void* m, int64_t ld) const
    {
        return load8<T, V>((const T*)m + row * ld, chunk(i), mask[i]);
    }
    __device__ __forceinline__ void saved(int i, bool matrix, float factor, float* v) const
    {
        if (matrix) {
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = whole[i].at(j) * factor;
        } else {
            ckpt_values<V>(codes[i], factor, v);
        }
    }
    __device__ __forceinline__ void stream(int i, float f, float* v) const { saved(i, p.stream, f, v); }
    __device__ __forceinline__ void block(int i, float f, float* v) const { saved(i, p.block, f, v); }
};

template <class T, bool V, int C>
__global__ void __launch_bounds__(1024) norm_backward_kernel(const NormBackParams p)
{
    pdl_enter();
    __shared__ float slots[2][32];
    int turn = 0;
    uint32_t mask[C];
#pragma unroll
    for (int i = 0; i < C; ++i) mask[i] = chunk_mask<V>((int64_t)i * blockDim.x + threadIdx.x, p.c.cols);
    const Columns<T, V, false> cols{p.c, nullptr};
    float sum_pre[C][8] = {}, sum_q[C][8] = {};
    float sum_scalar = 0.0f;
    for (int64_t row = blockIdx.x; row < p.c.rows; row += gridDim.x) {
        DirectLoader<T, V, C> in{p, mask, row};
        back_row<T, V, C, false>(p, row, in, mask, cols, sum_pre, sum_q, sum_scalar, slots, turn);
    }
    store_sums<V, C>(p, mask, sum_pre, sum_q, sum_scalar);
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
        const unsigned threads = (unsigned)((p.c.cols + 511) / 512) * 32;
        const size_t per_thread = 2 * (2 * 32 + (size_t)kItems<T> * sizeof(T) * 8);
        auto kernel = norm_backward_queue_kernel<T, kItems<T>>;
        e = cudaFuncSetAttribute((const void*)kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 (int)(per_thread * kQueueThreads));
        if (e == cudaSuccess) e = launch_kernel(kernel, grid, threads, per_thread * threads, s, p);
    } else if (p.c.vec) {
        e = launch_kernel(norm_backward_kernel<T, true, 4>, grid, (unsigned)((groups + 3) / 4) * 32, 0, s, p);
    } else if (groups <= 32) {
        e = launch_kernel(norm_backward_kernel<T, false, 1>, grid, (unsigned)groups * 32, 0, s, p);
    } else if (groups <= 64) {
        e = launch_kernel(norm_backward_kernel<T, false, 2>, grid, (unsigned)((groups + 1) / 2) * 32, 0, s, p);
    } else {
        e = launch_kernel(norm_backward_kernel<T, false, 4>, grid, (unsigned)((groups + 3) / 4) * 32, 0, s, p);
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
