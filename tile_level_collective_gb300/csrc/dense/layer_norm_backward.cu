// The backward pass of layer norm, with the reduction of the weight's and the
// bias' gradients over the rows.
//
// Bound by HBM: per element it reads dy, s and du and writes dx. One wave of
// blocks walks the rows with both column sums in registers and copies of the next
// rows queued in shared memory; one exchange of two sums per row. Each block
// writes its column sums as a partial row, and a second launch adds those in
// order (about 5 us). A short batch takes one launch, whose blocks for the column
// sums read the inputs again.
//
// Measured on GB300 (bf16, both launches, of 6.8 TB/s copied): 16384 x 8192 with
// du 181 us (5.9 TB/s; straight from memory 243), without 160; 8192 x 4096 56 and
// 50 us; f32 88 and 70 us (6.1 TB/s); 8192 x 4095 63 and 56 us. With 16-bit elements
// latency at 16 warps per SM, which 125 registers allow: half of the issue slots. Wide
// rows: 4096 x 16384 184 us.
#include "layers/layers_common.cuh"
#include "dense/dense_internal.h"
#include "host/host_checks.h"

namespace ptoc {

namespace {

// Where the weight's columns come from: binary32 copies that the thread keeps in
// shared memory (KEEP), or memory.
template <class T, int G, int C, bool KEEP>
struct Weight {
    const LayerNormBackParams& p;
    const int32_t (&col)[C];
    const uint32_t (&mask)[C];
    uint32_t kept;                          // [C][2][32] 16-byte words of the warp, from this lane's on

    __device__ __forceinline__ F8 load(int i) const
    {
        return load_param8<T, G>(p.weight, p.param_f32, col[i], mask[i]);
    }
    __device__ __forceinline__ uint32_t word(int n) const { return kept + (uint32_t)n * 512; }
    __device__ __forceinline__ void keep(int i) const
    {
        const F8 f = load(i);
#pragma unroll
        for (int h = 0; h < 2; ++h)
            asm volatile("st.shared.v2.u64 [%0], {%1, %2};" ::"r"(word(2 * i + h)), "l"(f.p[2 * h]), "l"(f.p[2 * h + 1])
                         : "memory");
    }
    __device__ __forceinline__ F8 columns(int i) const
    {
        if constexpr (!KEEP) return load(i);
        F8 f;
#pragma unroll
        for (int h = 0; h < 2; ++h)
            asm volatile("ld.shared.v2.u64 {%0, %1}, [%2];" : "=l"(f.p[2 * h]), "=l"(f.p[2 * h + 1])
                         : "r"(word(2 * i + h)) : "memory");
        return f;
    }
};

// One row. The loader gives, in this order, the statistics, the stream, dy, and
// du (if p.du), chunk by chunk. SUMS: the column sums are taken here.
template <class T, int G, int C, bool KEEP, bool SUMS, class Loader>
__device__ __forceinline__ void back_row(const LayerNormBackParams& p, int64_t row, Loader& in,
                                         const Weight<T, G, C, KEEP>& weight, F8 (&sum_w)[SUMS ? C : 1],
                                         F8 (&sum_b)[SUMS ? C : 1], SumSlots<2>& sums)
{
    const int32_t (&col)[C] = weight.col;
    const uint32_t (&mask)[C] = weight.mask;
    const float2 at = in.begin_row(row);
    const Pair shift = both(-at.x), scale = both(at.y);
    F8 n[C], t[C];
#pragma unroll
    for (int i = 0; i < C; ++i) {
        n[i] = in.matrix(i).expand();
#pragma unroll
        for (int j = 0; j < 4; ++j) n[i].p[j] = mul2(add2(n[i].p[j], shift), scale);
    }
    in.begin_dy();
    Pair s1[2] = {}, s2[2] = {};
#pragma unroll
    for (int i = 0; i < C; ++i) {
        t[i] = in.matrix(i).expand();
        const F8 w = weight.columns(i);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if constexpr (SUMS) {
                sum_b[i].p[j] = add2(sum_b[i].p[j], t[i].p[j]);
                sum_w[i].p[j] = fma2(t[i].p[j], n[i].p[j], sum_w[i].p[j]);
            }
            t[i].p[j] = mul2(t[i].p[j], w.p[j]);         // (zero past the row's end, where dy is)
            s1[j & 1] = add2(s1[j & 1], t[i].p[j]);
            s2[j & 1] = fma2(t[i].p[j], n[i].p[j], s2[j & 1]);
        }
    }
    float total[2] = {sum_of(add2(s1[0], s1[1])), sum_of(add2(s2[0], s2[1]))};
    sums.begin(total);
    in.begin_du();
    sums.end(total);
    const Pair m1 = both(-total[0] * p.inv_cols), m2 = both(-total[1] * p.inv_cols);
#pragma unroll
    for (int i = 0; i < C; ++i) {
        F8 carry = {};
        if (p.du) carry = in.matrix(i).expand();
#pragma unroll
        for (int j = 0; j < 4; ++j)
            t[i].p[j] = fma2(scale, fma2(m2, n[i].p[j], add2(t[i].p[j], m1)), carry.p[j]);
        store8<T, G>((T*)p.dx + row * p.ld_dx, col[i], mask[i], t[i]);
    }
    in.end_row();
}

// This block's partial rows of the column sums.
template <int G, int C>
__device__ __forceinline__ void store_sums(const LayerNormBackParams& p, const int32_t (&col)[C],
                                           const uint32_t (&mask)[C], const F8 (&sum_w)[C], const F8 (&sum_b)[C])
{
    const int64_t plane = (int64_t)gridDim.x * p.cols;
    float* mine = p.partial + (int64_t)blockIdx.x * p.cols;
#pragma unroll
    for (int i = 0; i < C; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            float a[2], b[2];
            split(sum_w[i].p[j / 2], a[0], a[1]);
            split(sum_b[i].p[j / 2], b[0], b[1]);
            if (mask[i] >> (j / G) & 1) {
                float* at = mine + col[i] + j / G * 32 * G + j % G;
                if (p.d_weight) at[0] = a[j & 1];
                if (p.d_bias) at[plane] = b[j & 1];
            }
        }
}

// Chunks straight from memory.
template <class T, int G, int C>
struct DirectLoader {
    const LayerNormBackParams& p;
    const int32_t (&col)[C];
    const uint32_t (&mask)[C];
    int64_t row;
    Raw8<T, G> whole[C];

    __device__ __forceinline__ void fetch(const void* m, int64_t ld)
    {
#pragma unroll
        for (int i = 0; i < C; ++i) whole[i] = load8<T, G>((const T*)m + row * ld, col[i], mask[i]);
    }
    __device__ __forceinline__ float2 begin_row(int64_t)
    {
        fetch(p.s, p.ld_s);
        return make_float2(p.stats[row], p.stats[p.rows + row]);
    }
    __device__ __forceinline__ void begin_dy() { fetch(p.dy, p.ld_dy); }
    __device__ __forceinline__ void begin_du()
    {
        if (p.du) fetch(p.du, p.ld_du);
    }
    __device__ __forceinline__ void end_row() {}
    __device__ __forceinline__ const Raw8<T, G>& matrix(int i) const { return whole[i]; }
};

// Rows of up to 8,192 columns with the column sums in registers (NARROW), and
// wider ones, for which layer_norm_columns_kernel takes them.
template <class T, int G, int C, bool NARROW>
__global__ void __launch_bounds__(NARROW ? 512 : 1024, 1) layer_norm_backward_kernel(const LayerNormBackParams p)
{
    pdl_enter();
    __shared__ __align__(16) float slots[2 * 2 * 32];
    SumSlots<2> sums(slots);
    int32_t col[C];
    uint32_t mask[C];
#pragma unroll
    for (int i = 0; i < C; ++i) {
        col[i] = first_col<G, C>(i);
        mask[i] = runs_below<G>(col[i], p.cols);
    }
    const Weight<T, G, C, false> weight{p, col, mask, 0};
    F8 sum_w[NARROW ? C : 1] = {}, sum_b[NARROW ? C : 1] = {};
    for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
        DirectLoader<T, G, C> in{p, col, mask, row};
        back_row<T, G, C, false, NARROW>(p, row, in, weight, sum_w, sum_b, sums);
    }
    if constexpr (NARROW) store_sums<G, C>(p, col, mask, sum_w, sum_b);
}

// A warp's column sums of 256 columns from `first` on, of the rows row0, row0 + step, ...
template <class T, int G, int WARPS>
__device__ __forceinline__ void sum_columns(const LayerNormBackParams& p, int32_t first, int64_t row0, int64_t step,
                                            float (&sums)[WARPS][2][256])
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int32_t col = first + lane * G;
    const uint32_t mask = runs_below<G>(col, p.cols);
    F8 sum_w = {}, sum_b = {};
#pragma unroll 4
    for (int64_t row = row0; row < p.rows; row += step) {
        const Pair shift = both(-p.stats[row]), scale = both(p.stats[p.rows + row]);
        const F8 s = load8<T, G>((const T*)p.s + row * p.ld_s, col, mask).expand();
        const F8 dy = load8<T, G>((const T*)p.dy + row * p.ld_dy, col, mask).expand();
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            sum_w.p[j] = fma2(dy.p[j], mul2(add2(s.p[j], shift), scale), sum_w.p[j]);
            sum_b.p[j] = add2(sum_b.p[j], dy.p[j]);
        }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        float a[2], b[2];
        split(sum_w.p[j / 2], a[0], a[1]);
        split(sum_b.p[j / 2], b[0], b[1]);
        const int at = lane * G + j / G * 32 * G + j % G;
        sums[warp][0][at] = a[j & 1];
        sums[warp][1][at] = b[j & 1];
    }
}

constexpr int kColumnWarps = 8;

// The column sums of wide rows, which read the stream and dy a second time (in
// registers beside the row they would spill: 4096 x 16384 bf16 1080 us): a block takes
// 256 columns of the rows that block y of the row kernel's grid would; its warps
// take rows in turn and are added in order.
template <class T, int G>
__global__ void __launch_bounds__(kColumnWarps * 32) layer_norm_columns_kernel(const LayerNormBackParams p)
{
    pdl_enter();
    __shared__ float sums[kColumnWarps][2][256];
    const int32_t first = (int32_t)blockIdx.x * 256;
    sum_columns<T, G, kColumnWarps>(p, first, blockIdx.y + (int64_t)(threadIdx.x >> 5) * p.grid,
                                    (int64_t)kColumnWarps * p.grid, sums);
    __syncthreads();
    if (first + (int)threadIdx.x >= p.cols) return;
    const int64_t plane = (int64_t)p.grid * p.cols;
    float* to = p.partial + (int64_t)blockIdx.y * p.cols + first + threadIdx.x;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        float sum = 0.0f;
#pragma unroll
        for (int w = 0; w < kColumnWarps; ++w) sum += sums[w][k][threadIdx.x];
        if (k ? p.d_bias : p.d_weight) to[k * plane] = sum;
    }
}

// Chunks from the thread's queue of K items, in the order of their use: the
// stream, dy and (with it) du of this row and of the next ones. The rows' two
// statistics are read a row before their use.
template <class T, int C, int K, bool ODD>
struct QueueLoader {
    using Q = Queue<T, C, K, ODD>;
    static constexpr int G = Q::G;
    const LayerNormBackParams& p;
    Q queue;
    const int32_t (&col)[C];
    const uint32_t (&mask)[C];
    int64_t ahead;                          // the row whose items are copied next
    const T *s_row, *dy_row, *du_row;       // in that row
    int item = 0;                           // 0: its stream, 1: dy, 2: du
    uint32_t shift = 0, row = 0;            // where the current item's row begins in its words
    float2 next;

    __device__ __forceinline__ QueueLoader(const LayerNormBackParams& q, unsigned char* smem, const int32_t (&c)[C],
                                           const uint32_t (&m)[C])
        : p(q), queue(smem, m), col(c), mask(m), ahead(blockIdx.x)
    {
        const int64_t r = blockIdx.x;
        s_row = (const T*)p.s + r * p.ld_s;
        dy_row = (const T*)p.dy + r * p.ld_dy;
        du_row = (const T*)p.du + r * p.ld_du;
        next = stats_of(r);
#pragma unroll 1
        for (int i = 0; i < K; ++i) push();
    }
    __device__ __forceinline__ float2 stats_of(int64_t r) const
    {
        return r < p.rows ? make_float2(p.stats[r], p.stats[p.rows + r]) : make_float2(0.0f, 0.0f);
    }
    __device__ __forceinline__ void push()
    {
        queue.done();
        if (ahead < p.rows) {
            queue.copy_row(item == 0 ? s_row : item == 1 ? dy_row : du_row, col, mask, p.cols);
            if (++item == 2 + (p.du != nullptr)) {
                item = 0;
                ahead += gridDim.x;
                s_row += p.step_s;
                dy_row += p.step_dy;
                du_row += p.step_du;
            }
        }
        queue.next();
    }
    __device__ __forceinline__ void begin(int64_t ld)
    {
        queue.wait();
        if constexpr (ODD) shift = row * (uint32_t)ld * (uint32_t)sizeof(T) & 15u;
    }
    __device__ __forceinline__ float2 begin_row(int64_t r)
    {
        const float2 now = next;
        next = stats_of(r + gridDim.x);
        row = (uint32_t)r;
        begin(p.ld_s);
        return now;
    }
    __device__ __forceinline__ void begin_dy()
    {
        push();
        begin(p.ld_dy);
    }
    __device__ __forceinline__ void begin_du()
    {
        if (!p.du) return;
        push();
        begin(p.ld_du);
    }
    __device__ __forceinline__ void end_row() { push(); }
    __device__ __forceinline__ Raw8<T, G> matrix(int i) const { return queue.chunk(i, shift); }
};

constexpr int kQueueThreads = 512;
template <class T>
constexpr int kQueueItems = 10 / ((int)sizeof(T) / 2);       // 160 KiB on an SM, beside the weight's 32

template <class T, bool ODD>
__global__ void __launch_bounds__(kQueueThreads, 1) layer_norm_backward_queue_kernel(const LayerNormBackParams p)
{
    constexpr int C = 2, G = ODD ? 1 : kVector<T>;
    pdl_enter();
    extern __shared__ __align__(16) unsigned char smem[];
    __shared__ __align__(16) float slots[2 * 2 * 32];
    SumSlots<2> sums(slots);
    int32_t col[C];
    uint32_t mask[C];
#pragma unroll
    for (int i = 0; i < C; ++i) {
        col[i] = first_col<G, C>(i);
        mask[i] = runs_below<G>(col[i], p.cols);
    }
    QueueLoader<T, C, kQueueItems<T>, ODD> in(p, smem + (size_t)blockDim.x * C * 32, col, mask);
    const uint32_t kept = (uint32_t)__cvta_generic_to_shared(smem) + (threadIdx.x >> 5) * (C * 1024);
    const Weight<T, G, C, true> weight{p, col, mask, kept + (threadIdx.x & 31) * 16};
#pragma unroll
    for (int i = 0; i < C; ++i) weight.keep(i);
    F8 sum_w[C] = {}, sum_b[C] = {};
    for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x)
        back_row<T, G, C, true, true>(p, row, in, weight, sum_w, sum_b, sums);
    asm volatile("cp.async.wait_all;" ::: "memory");
    store_sums<G, C>(p, col, mask, sum_w, sum_b);
}

// A short batch in one launch: the first blocks take a row each, the others 256
// columns of all rows, from the inputs: their sums do not wait for the rows'
// blocks. (dx is then neither dy nor the stream.)
constexpr int kShortThreads = 512;

template <class T, int G>
__global__ void __launch_bounds__(kShortThreads, 1) layer_norm_backward_short_kernel(const LayerNormBackParams p)
{
    pdl_enter();
    if (blockIdx.x < p.rows) {
        constexpr int C = 2;
        __shared__ __align__(16) float slots[2 * 2 * 32];
        SumSlots<2> sums(slots);
        int32_t col[C];
        uint32_t mask[C];
#pragma unroll
        for (int i = 0; i < C; ++i) {
            col[i] = first_col<G, C>(i);
            mask[i] = runs_below<G>(col[i], p.cols);
        }
        const Weight<T, G, C, false> weight{p, col, mask, 0};
        F8 none_w[1], none_b[1];
        DirectLoader<T, G, C> in{p, col, mask, blockIdx.x};
        back_row<T, G, C, false, false>(p, blockIdx.x, in, weight, none_w, none_b, sums);
        return;
    }
    constexpr int kWarps = kShortThreads / 32;
    __shared__ float sums[kWarps][2][256];
    const int first = (int)(blockIdx.x - p.rows) * 256;
    sum_columns<T, G, kWarps>(p, first, (int)threadIdx.x >> 5, kWarps, sums);
    __syncthreads();
    const int which = (int)threadIdx.x >> 8, at = (int)threadIdx.x & 255;
    float* to = which ? p.d_bias : p.d_weight;
    if (!to || first + at >= p.cols) return;
    float sum = 0.0f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) sum += sums[w][which][at];
    to[first + at] = sum;
}

constexpr int kSumThreads = 1024;

// Sums of the partial rows: a block takes 32 columns of the weight's (y = 0) or
// the bias' gradient; its 32 warps each add a run of the partial rows in order,
// and the runs are added in order.
__global__ void __launch_bounds__(kSumThreads) layer_norm_sum_kernel(const LayerNormBackParams p)
{
    pdl_enter();
    __shared__ float runs[kSumThreads / 32][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t col = (int64_t)blockIdx.x * 32 + lane;
    float* to = blockIdx.y ? p.d_bias : p.d_weight;
    const bool live = to && col < p.cols;
    float sum = 0.0f;
    if (live) {
        const float* src = p.partial + (int64_t)blockIdx.y * p.grid * p.cols + col;
        const int per = (p.grid + kSumThreads / 32 - 1) / (kSumThreads / 32);
        const int end = min(p.grid, (warp + 1) * per);
#pragma unroll 8
        for (int b = warp * per; b < end; ++b) sum += src[b * p.cols];
    }
    runs[warp][lane] = sum;
    __syncthreads();
    if (warp || !live) return;
    sum = 0.0f;
#pragma unroll
    for (int w = 0; w < kSumThreads / 32; ++w) sum += runs[w][lane];
    to[col] = sum;
}

// Rows from memory. The sums of wide rows come first: dx may lie over dy.
template <class T, int G>
cudaError_t launch_direct(const LayerNormBackParams& p, cudaStream_t s)
{
    const int64_t groups = (p.cols + 255) / 256;
    const unsigned by2 = (unsigned)((groups + 1) / 2) * 32, by4 = (unsigned)((groups + 3) / 4) * 32;
    const dim3 grid((unsigned)p.grid);
    if (groups <= 32) return launch_kernel(layer_norm_backward_kernel<T, G, 2, true>, grid, by2, 0, s, p);
    if (p.d_weight || p.d_bias) {
        const cudaError_t e = launch_kernel(layer_norm_columns_kernel<T, G>, dim3((unsigned)groups, (unsigned)p.grid),
                                            kColumnWarps * 32, 0, s, p);
        if (e != cudaSuccess) return e;
    }
    if (groups <= 64) return launch_kernel(layer_norm_backward_kernel<T, G, 2, false>, grid, by2, 0, s, p);
    return launch_kernel(layer_norm_backward_kernel<T, G, 4, false>, grid, by4, 0, s, p);
}

// Shared memory of a block: the weight's columns and the queues.
template <class T, bool ODD>
constexpr size_t queue_bytes(size_t threads)
{
    return threads * 2 * 32 + Queue<T, 2, kQueueItems<T>, ODD>::bytes(threads);
}

template <class T, bool ODD>
cudaError_t launch_queue(const LayerNormBackParams& p, cudaStream_t s)
{
    const unsigned threads = (unsigned)((p.cols + 511) / 512) * 32;
    auto kernel = layer_norm_backward_queue_kernel<T, ODD>;
    static std::atomic<uint64_t> done{0};
    LayerNormBackParams q = p;
    q.step_s = (int64_t)p.grid * p.ld_s;
    q.step_dy = (int64_t)p.grid * p.ld_dy;
    q.step_du = (int64_t)p.grid * p.ld_du;
    return launch_shared((const void*)kernel, (int)queue_bytes<T, ODD>(kQueueThreads), done, [&] {
        return launch_kernel(kernel, dim3((unsigned)p.grid), threads, queue_bytes<T, ODD>(threads), s, q);
    });
}

// Up to this many rows one launch that reads the inputs twice takes less than two.
// In a graph, us (one launch, two), bf16: 16 x 1000 2.5, 4.7; 128 x 256 3.5, 4.8;
// 128 x 8192 5.2, 18; 256 x 256 6.0, 4.7. With more columns more blocks share the sums:
// 512 x 2048 11, 18; 512 x 8192 12, 23; f32 512 x 2048 12, 12.4; 512 x 1000 12, 8.2;
// but element by element, at odd pitches, 512 x 2048 22, 8.5 (128 x 2048 5.4, 5.6). 1024 x 4096 bf16 is
// 20 either way.
inline int64_t short_rows(const LayerNormBackParams& p) { return p.access == kAligned && p.cols >= 2048 ? 512 : 128; }

template <class T, int G>
cudaError_t launch_short(const LayerNormBackParams& p, cudaStream_t s)
{
    const unsigned columns = p.d_weight || p.d_bias ? (unsigned)((p.cols + 255) / 256) : 0;
    return launch_kernel(layer_norm_backward_short_kernel<T, G>, dim3((unsigned)p.rows + columns), kShortThreads, 0, s,
                         p);
}

template <class T>
cudaError_t launch(const LayerNormBackParams& p, cudaStream_t s)
{
    const bool narrow = p.cols <= kQueueThreads * 16;
    if (narrow && p.rows <= short_rows(p) && p.dx != p.dy)
        return p.access == kAligned ? launch_short<T, kVector<T>>(p, s) : launch_short<T, 1>(p, s);
    const cudaError_t e = narrow && p.access == kAligned    ? launch_queue<T, false>(p, s)
                          : narrow && p.access == kOddPitch ? launch_queue<T, true>(p, s)
                          : p.access == kAligned            ? launch_direct<T, kVector<T>>(p, s)
                                                            : launch_direct<T, 1>(p, s);
    if (e != cudaSuccess || (!p.d_weight && !p.d_bias)) return e;
    return launch_kernel(layer_norm_sum_kernel, dim3((unsigned)((p.cols + 31) / 32), 2), kSumThreads, 0, s, p);
}

}  // namespace

// One wave: the blocks that 512 threads of two chunks on each SM make up. The
// count is GB300's, not the device's answer: the order of the sums and the
// workspace then depend on the sizes alone.
int layer_norm_backward_grid(int64_t rows, int64_t cols)
{
    constexpr int kSms = 152;
    const int64_t threads = (cols + 511) / 512 * 32;
    const int64_t per_sm = threads >= 512 ? 1 : 512 / threads < 12 ? 512 / threads : 12;
    const int64_t most = (int64_t)kSms * per_sm;
    return (int)(rows < most ? rows : most);
}

cudaError_t launch_layer_norm_backward(const LayerNormBackParams& p, int dtype, cudaStream_t s)
{
    switch (dtype) {
    case PTOC_F32: return launch<float>(p, s);
    case PTOC_F16: return launch<__half>(p, s);
    default: return launch<__nv_bfloat16>(p, s);
    }
}

}  // namespace ptoc
