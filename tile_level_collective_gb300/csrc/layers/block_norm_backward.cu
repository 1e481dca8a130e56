// The backward pass of the norms around a block.
//
// With st = s * r, ah = a * ra, and gw the columns' factor (the weight of the
// norm after the block, times branch_scale and the gate where that varies
// along the columns; F is the rest, one number for the row):
//   ds = v - r * m * st,  v = du + r * wpre * dy,  m = mean(wpre * dy * st)
//   d_residual = residual_scale * ds
//   t = gw * ds;  d_block = ra * F * (t - ah * mean(t * ah))
// The second mean is mean(gw * ah * v) - r * m * mean(gw * ah * st), so one
// block-wide exchange of three sums serves both (with two, one after the
// other, 8192 x 4096 from checkpoints took 81 us, and 16384 x 8192 274).
// The weights' and the gate's gradients need two sums over the rows for each
// column: of dy * st, and Q of ds * ah (times the gate where it varies by
// row), from which d_post_weight and the gate's gradient follow.
//
// Bound by HBM: per element it reads dy, du, s and a (the last two in 2 or 4
// bytes, or 33/32 as 8-bit checkpoints) and writes d_residual and d_block.
// One wave of blocks walks the rows with the two column sums in registers;
// copies of the next row are queued in shared memory, as in the forward pass.
// Each block writes its column sums as one partial row, and a second launch
// adds the partial rows in order (about 4 us).
//
// Measured on GB300 (bf16, both launches; of 6.79 TB/s copied): 8192 x 4096
// from checkpoints 71 us (4.8 TB/s), from matrices 77 us (5.2 TB/s), from
// checkpoints of 4095 columns 99 us; 16384 x 8192 from checkpoints 237 us (5.7
// TB/s); f32 8192 x 4096 136 us (5.9 TB/s). With 16-bit elements and codes
// instructions and their latency come before HBM: 580 instructions per thread
// and row of 16 columns, 50 % of the issue slots at 16 warps per SM, which the
// registers allow (two column sums, three arrays of the row: 120). One chunk
// per thread in 64 registers took 96 us, four chunks in 255 registers 104 us,
// where two took 81.
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

template <class T, int G>
__device__ __forceinline__ F8 gate8(const NormCommon& k, int64_t row, int32_t col, uint32_t mask)
{
    return load_param8<T, G>((const char*)k.gate + row * k.gate_rs * (k.param_f32 ? 4 : (int)sizeof(T)), k.param_f32,
                             col, mask);
}

// Where the per-column parameters of chunk i come from: f32 copies that the
// thread keeps in shared memory (KEEP), or memory.
template <class T, int G, int C, bool KEEP>
struct Columns {
    const NormCommon& k;
    const int32_t (&col)[C];
    const uint32_t (&mask)[C];
    uint32_t kept;                          // [2][C][2][32] 16-byte words of the warp: wpre, then the factor

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
    __device__ __forceinline__ uint32_t word(int n) const { return kept + (uint32_t)n * 512; }
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

// What a row has one of: its statistics, and the gate where it is one number.
struct RowScalars {
    float ra, r, gate;
};

// One row. The loader gives, in this order: what the row has one of, and chunk
// by chunk the stream times a factor, dy, du (if p.du), the block output times
// a factor. ELEMENT: the gate varies along both axes.
template <class T, int G, int C, bool KEEP, bool ELEMENT, class Loader>
__device__ __forceinline__ void back_row(const NormBackParams& p, int64_t row, Loader& in,
                                         const Columns<T, G, C, KEEP>& cols, F8 (&sum_pre)[C], F8 (&sum_q)[C],
                                         float& sum_scalar, SumSlots<3>& sums)
{
    const NormCommon& k = p.c;
    const int32_t (&col)[C] = cols.col;
    const uint32_t (&mask)[C] = cols.mask;
    const RowScalars at = in.begin_row(row);
    F8 st[C], v[C], ah[C];
    Pair s1 = 0, s2 = 0, s3 = 0;
#pragma unroll
    for (int i = 0; i < C; ++i) st[i] = in.stream(i, at.r);
    in.end_stream();
    in.begin_dy();
#pragma unroll
    for (int i = 0; i < C; ++i) {
        const F8 dy = in.matrix(i).expand(), w = cols.pre(i);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            v[i].p[j] = mul2(w.p[j], dy.p[j]);
            sum_pre[i].p[j] = fma2(dy.p[j], st[i].p[j], sum_pre[i].p[j]);
            s1 = fma2(v[i].p[j], st[i].p[j], s1);
        }
    }
    in.end_dy();
    in.begin_du();
    const Pair r2 = both(at.r);
    if (p.du) {
#pragma unroll
        for (int i = 0; i < C; ++i) {
            const F8 du = in.matrix(i).expand();
#pragma unroll
            for (int j = 0; j < 4; ++j) v[i].p[j] = fma2(r2, v[i].p[j], du.p[j]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < C; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) v[i].p[j] = mul2(r2, v[i].p[j]);
    }
    in.end_du();
    in.begin_block();
#pragma unroll
    for (int i = 0; i < C; ++i) ah[i] = in.block(i, at.ra);
    in.end_block();
    F8 g[ELEMENT ? C : 1];
#pragma unroll
    for (int i = 0; i < C; ++i) {
        F8 w = cols.factor(i);
        if constexpr (ELEMENT) {
            g[i] = gate8<T, G>(k, row, col[i], mask[i]);
#pragma unroll
            for (int j = 0; j < 4; ++j) w.p[j] = mul2(w.p[j], mul2(both(k.branch_scale), g[i].p[j]));
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const Pair wa = mul2(w.p[j], ah[i].p[j]);
            s2 = fma2(wa, v[i].p[j], s2);
            s3 = fma2(wa, st[i].p[j], s3);
        }
    }
    float total[3] = {sum_of(s1), sum_of(s2), sum_of(s3)};
    sums.sum(total);
    const float rm = at.r * (total[0] * k.inv_cols);
    const float dot = total[1] - rm * total[2];             // of gw * ds and ah
    if (p.gate_kind == kGateToken || p.gate_kind == kGateScalar) {
        const float d = k.branch_scale * dot;
        if (p.gate_kind == kGateToken && threadIdx.x == 0) p.d_gate[row] = d;
        sum_scalar += d;
    }
    const bool by_column = k.gate_cs != 0;
    const bool q_scaled = !by_column && k.gate_rs;          // a gate that varies by row goes into Q
    const Pair m1 = both(-rm), m2 = both(k.post_norm ? -dot * k.inv_cols : 0.0f);
    const Pair f = both(at.ra * (by_column ? 1.0f : k.branch_scale * at.gate)), keep = both(k.residual_scale);
    T* d_residual = (T*)p.d_residual + row * p.ld_dres;
    T* d_block = (T*)p.d_block + row * p.ld_dblk;
#pragma unroll
    for (int i = 0; i < C; ++i) {
        F8 out, w = cols.factor(i);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            v[i].p[j] = fma2(m1, st[i].p[j], v[i].p[j]);    // ds
            out.p[j] = mul2(keep, v[i].p[j]);
        }
        store8<T, G>(d_residual, col[i], mask[i], out);
        if constexpr (ELEMENT) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                float e[2];
                const Pair d = mul2(both(k.branch_scale), mul2(v[i].p[j / 2], mul2(ah[i].p[j / 2], w.p[j / 2])));
                split(d, e[0], e[1]);
                // packed rows of floats, whose alignment follows the number of columns
                if (p.gate_kind == kGateElement && (mask[i] >> (j / G) & 1))
                    p.d_gate[row * k.cols + col[i] + j / G * 32 * G + j % G] = e[j & 1];
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                sum_q[i].p[j] = fma2(mul2(g[i].p[j], v[i].p[j]), ah[i].p[j], sum_q[i].p[j]);
                w.p[j] = mul2(w.p[j], mul2(both(k.branch_scale), g[i].p[j]));
            }
        } else if (q_scaled) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                sum_q[i].p[j] = fma2(mul2(both(at.gate), v[i].p[j]), ah[i].p[j], sum_q[i].p[j]);
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) sum_q[i].p[j] = fma2(v[i].p[j], ah[i].p[j], sum_q[i].p[j]);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) out.p[j] = mul2(f, fma2(m2, ah[i].p[j], mul2(w.p[j], v[i].p[j])));
        store8<T, G>(d_block, col[i], mask[i], out);
    }
}

// This block's partial rows of the column sums.
template <int G, int C>
__device__ __forceinline__ void store_sums(const NormBackParams& p, const int32_t (&col)[C], const uint32_t (&mask)[C],
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

// What rows have one of, and the scales of the checkpoints' blocks, of
// kHeaderRows rows of this block at a time, in shared memory. Loaded for each
// row into registers they cost more, even a row ahead of their use: a warp has
// few counters for its loads, and shared-memory reads that follow a load wait
// for it too (8192 x 4096 from checkpoints: 93 us so, 81 in batches). A scale
// is a power of two (or NaN): the upper half of its binary32 form. Binary32
// rows of 8,192 columns at odd pitches have 199 KB of parameters and queues,
// which leaves room for 16 rows.
template <class T>
constexpr int kHeaderRowsOf = sizeof(T) == 4 ? 16 : 32;

template <int kHeaderRows>
struct Header {
    float4* values;                         // [kHeaderRows]: r, ra, gate
    uint16_t* scales;                       // [kHeaderRows][2][width]: the stream's, the block output's
    int blocks, width, turn;                // of a row; with those past its end up to the last warp's, zeros
    uint32_t mine;                          // this thread's first scale of the current row

    static constexpr size_t size(size_t threads) { return kHeaderRows * (16 + threads * 2); }
    template <int G>
    __device__ __forceinline__ Header(const NormCommon& k, unsigned char* smem, std::integral_constant<int, G>)
        : values((float4*)smem), scales((uint16_t*)(smem + kHeaderRows * 16)), blocks((int)((k.cols + 31) >> 5)),
          width((int)blockDim.x / 2), turn(kHeaderRows - 1),
          mine((uint32_t)__cvta_generic_to_shared(scales) +
               ((threadIdx.x >> 5) * 16 + (G == 1 ? 0 : (threadIdx.x & 31) * G / 32) + 2 * turn * width) * 2)
    {
        for (int i = threadIdx.x; i < kHeaderRows * width; i += blockDim.x) ((uint32_t*)scales)[i] = 0;
    }
    // Go on to `row`, the next one of this block.
    template <class T, bool CKPT>
    __device__ __forceinline__ void advance(const NormBackParams& p, int64_t row)
    {
        mine += 4 * width;
        if (++turn < kHeaderRows) return;
        turn = 0;
        mine -= 4 * kHeaderRows * width;
        __syncthreads();                    // the rows before are done with theirs
        const int64_t left = (p.c.rows - 1 - row) / gridDim.x + 1;
        const uint32_t rows = left < kHeaderRows ? (uint32_t)left : kHeaderRows;
        if (threadIdx.x < rows) {
            const int64_t r = row + (int64_t)threadIdx.x * gridDim.x;
            values[threadIdx.x] = make_float4(p.rstd[p.c.rows + r], p.c.post_norm ? p.rstd[r] : 1.0f,
                                              gate_of_row<T>(p.c, r), 0.0f);
        }
        if constexpr (CKPT) {
            load_scales(0, p.stream_ckpt, row, rows);
            load_scales(1, p.block_ckpt, row, rows);
        }
        __syncthreads();
    }
    static __device__ __forceinline__ uint32_t scale_bits(uint32_t byte)
    {
        return __float_as_uint(ckpt_scale(byte)) >> 16;
    }
    // Words of four bytes where the checkpoint's rows allow them, several in
    // flight per thread: a batch costs about 1 us, byte by byte about 4.
    __device__ __forceinline__ void load_scales(int which, const ptoc_ckpt8& k, int64_t row, uint32_t rows)
    {
        uint16_t* to = scales + which * width;
        const uint32_t pitch = 2 * (uint32_t)width;
        const uint32_t words = (uint32_t)blocks / 4;
        if (words && words * 4 == (uint32_t)blocks && words <= blockDim.x &&
            (((uintptr_t)k.exps | (uintptr_t)k.ld_exps) & 3u) == 0) {
            constexpr int kAtOnce = 4;
            const uint32_t i0 = threadIdx.x / words, w = threadIdx.x - i0 * words, step = blockDim.x / words;
            if (i0 >= step) return;
            const uint8_t* from = k.exps + row * k.ld_exps + 4 * w;
            for (uint32_t i = i0; i < rows; i += kAtOnce * step) {
                uint32_t v[kAtOnce];
#pragma unroll
                for (int q = 0; q < kAtOnce; ++q)
                    v[q] = i + q * step < rows
                               ? *(const uint32_t*)(from + (int64_t)(i + q * step) * gridDim.x * k.ld_exps) : 0u;
#pragma unroll
                for (int q = 0; q < kAtOnce; ++q)
                    if (i + q * step < rows)
                        *(uint2*)(to + (i + q * step) * pitch + 4 * w) =
                            make_uint2(scale_bits(v[q] & 255u) | scale_bits(v[q] >> 8 & 255u) << 16,
                                       scale_bits(v[q] >> 16 & 255u) | scale_bits(v[q] >> 24) << 16);
            }
            return;
        }
        constexpr int kAtOnce = 8;
        for (uint32_t n0 = threadIdx.x; n0 < rows * blocks; n0 += kAtOnce * blockDim.x) {
            uint32_t byte[kAtOnce];
#pragma unroll
            for (int q = 0; q < kAtOnce; ++q) {
                const uint32_t n = n0 + q * blockDim.x, i = n / (uint32_t)blocks;
                byte[q] = n < rows * blocks ? k.exps[(row + (int64_t)i * gridDim.x) * k.ld_exps + (n - i * blocks)] : 0;
            }
#pragma unroll
            for (int q = 0; q < kAtOnce; ++q)
            {
                const uint32_t n = n0 + q * blockDim.x, i = n / (uint32_t)blocks;
                if (n < rows * blocks) to[i * pitch + (n - i * blocks)] = (uint16_t)scale_bits(byte[q]);
            }
        }
    }
    __device__ __forceinline__ RowScalars scalars() const
    {
        const float4 v = values[turn];
        return RowScalars{v.y, v.x, v.z};
    }
    // Of the block that is n after the thread's first one.
    __device__ __forceinline__ float scale(int which, int n) const
    {
        uint16_t h;
        asm volatile("ld.shared.u16 %0, [%1];" : "=h"(h) : "r"(mine + (which ? 2 * width : 0) + 2 * n) : "memory");
        return __uint_as_float((uint32_t)h << 16);
    }
};

// Chunks from the thread's queue. A row has four items: stream, dy, du (empty
// without du) and block. Each has a slot, which is filled with the next row's
// as soon as it has been read. CKPT: stream and block are checkpoints; else
// both are matrices.
template <class T, int C, bool CKPT, bool ODD>
struct QueueLoader {
    enum Item { kStream = 0, kDy = 1, kDu = 2, kBlockOut = 3 };
    using Q = Queue<T, C, 4, ODD>;
    static constexpr int G = Q::G;
    const NormBackParams& p;
    Q queue;
    const int32_t (&col)[C];
    const uint32_t (&mask)[C];
    int64_t ahead;                          // the row whose items are copied next
    bool more;                              // whether there is one
    const char *stream_row, *dy_row, *du_row, *block_row;               // in that row
    uint32_t shift;                         // where the current item's row begins in its words
    uint32_t row;
    Header<kHeaderRowsOf<T>> head;

    __device__ __forceinline__ QueueLoader(const NormBackParams& q, unsigned char* smem, const int32_t (&c)[C],
                                           const uint32_t (&m)[C])
        : p(q), queue(smem, m), col(c), mask(m), ahead(blockIdx.x), more(ahead < q.c.rows),
          head(q.c, smem + Q::bytes(blockDim.x), std::integral_constant<int, G>())
    {
        const int64_t row = blockIdx.x;
        stream_row = CKPT ? (const char*)(p.stream_ckpt.codes + row * p.stream_ckpt.ld_codes)
                          : (const char*)((const T*)p.stream + row * p.ld_stream);
        block_row = CKPT ? (const char*)(p.block_ckpt.codes + row * p.block_ckpt.ld_codes)
                         : (const char*)((const T*)p.block + row * p.ld_block);
        dy_row = (const char*)((const T*)p.dy + row * p.ld_dy);
        du_row = (const char*)((const T*)p.du + row * p.ld_du);
        end_stream();
        end_dy();
        end_du();
        end_block();
    }
    __device__ __forceinline__ RowScalars begin_row(int64_t row)
    {
        head.template advance<T, CKPT>(p, row);
        this->row = (uint32_t)row;
        begin(kStream, CKPT ? p.stream_ckpt.ld_codes : p.ld_stream, CKPT ? 1 : sizeof(T));
        return head.scalars();
    }
    // The next item: wait for it.
    __device__ __forceinline__ void begin(Item item, int64_t ld, uint32_t size)
    {
        queue.go(item);
        queue.wait();
        if constexpr (ODD) shift = row * (uint32_t)ld * size & 15u;
    }
    // An item is read: its slot takes the next of its kind.
    __device__ __forceinline__ void push(Item item, const char*& at, int64_t step)
    {
        queue.go(item);
        queue.done();
        if (more) {
            if (CKPT && (item == kStream || item == kBlockOut))
                queue.copy_codes((const int8_t*)at, col, mask, p.c.cols);
            else
                queue.copy_row((const T*)at, col, mask, p.c.cols);
            at += step;
        }
        queue.commit();
    }
    __device__ __forceinline__ void end_stream() { push(kStream, stream_row, p.step_stream); }
    __device__ __forceinline__ void end_dy() { push(kDy, dy_row, p.step_dy); }
    __device__ __forceinline__ void end_du()
    {
        if (p.du) push(kDu, du_row, p.step_du);
        else queue.commit();
    }
    __device__ __forceinline__ void end_block()
    {
        push(kBlockOut, block_row, p.step_block);
        ahead += gridDim.x;
        more = ahead < p.c.rows;
    }
    __device__ __forceinline__ void begin_dy() { begin(kDy, p.ld_dy, sizeof(T)); }
    __device__ __forceinline__ void begin_du() { begin(kDu, p.ld_du, sizeof(T)); }
    __device__ __forceinline__ void begin_block()
    {
        begin(kBlockOut, CKPT ? p.block_ckpt.ld_codes : p.ld_block, CKPT ? 1 : sizeof(T));
    }
    __device__ __forceinline__ Raw8<T, G> matrix(int i) const { return queue.chunk(i, shift); }
    __device__ __forceinline__ F8 saved(int i, int which, float factor) const
    {
        F8 f;
        if constexpr (CKPT) {
            uint32_t w[ODD ? 8 : 2];
            queue.codes(i, shift, w);
            constexpr int kRuns = 8 / G;
            float scale[kRuns];
#pragma unroll
            for (int q = 0; q < kRuns; ++q) scale[q] = head.scale(which, 8 * i + q * G) * factor;
            Pair by[ODD ? 4 : kRuns];
#pragma unroll
            for (int q = 0; q < (ODD ? 4 : kRuns); ++q)
                by[q] = ODD ? pair(scale[2 * q % kRuns], scale[(2 * q + 1) % kRuns]) : both(scale[q]);
            f = code_values<G>(w, by);
        } else {
            f = queue.chunk(i, shift).expand();
#pragma unroll
            for (int j = 0; j < 4; ++j) f.p[j] = mul2(f.p[j], both(factor));
        }
        return f;
    }
    __device__ __forceinline__ F8 stream(int i, float f) const { return saved(i, 0, f); }
    __device__ __forceinline__ F8 block(int i, float f) const { return saved(i, 1, f); }
};

constexpr int kQueueThreads = 512;

template <class T, bool CKPT, bool ODD>
__global__ void __launch_bounds__(kQueueThreads) norm_backward_queue_kernel(const NormBackParams p)
{
    constexpr int C = 2, G = ODD ? 1 : kVector<T>;
    pdl_enter();
    extern __shared__ __align__(16) unsigned char smem[];
    __shared__ __align__(16) float slots[2 * 3 * 32];
    SumSlots<3> sums(slots);
    int32_t col[C];
    uint32_t mask[C];
#pragma unroll
    for (int i = 0; i < C; ++i) {
        col[i] = first_col<G, C>(i);
        mask[i] = runs_below<G>(col[i], p.c.cols);
    }
    QueueLoader<T, C, CKPT, ODD> in(p, smem + (size_t)blockDim.x * C * 64, col, mask);
    const uint32_t kept = (uint32_t)__cvta_generic_to_shared(smem) + (threadIdx.x >> 5) * (C * 2048);
    const Columns<T, G, C, true> cols{p.c, col, mask, kept + (threadIdx.x & 31) * 16};
    const Columns<T, G, C, false> memory{p.c, col, mask, 0};
#pragma unroll
    for (int i = 0; i < C; ++i) {
        cols.keep(2 * i, memory.pre(i));
        cols.keep(2 * (C + i), memory.load_factor(i));
    }
    F8 sum_pre[C] = {}, sum_q[C] = {};
    float sum_scalar = 0.0f;
    for (int64_t row = blockIdx.x; row < p.c.rows; row += gridDim.x) {
        back_row<T, G, C, true, false>(p, row, in, cols, sum_pre, sum_q, sum_scalar, sums);
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    store_sums<G, C>(p, col, mask, sum_pre, sum_q, sum_scalar);
}

// Chunks straight from memory, for rows at any address and very wide ones.
template <class T, int G, int C>
struct DirectLoader {
    const NormBackParams& p;
    const int32_t (&col)[C];
    const uint32_t (&mask)[C];
    int64_t row;
    CkptRaw<G> codes[C];
    Raw8<T, G> whole[C];

    __device__ __forceinline__ void end_stream() {}
    __device__ __forceinline__ void end_dy() {}
    __device__ __forceinline__ void end_du() {}
    __device__ __forceinline__ void end_block() {}
    __device__ __forceinline__ void fetch(const void* m, int64_t ld, const ptoc_ckpt8& k)
    {
        const Ckpt c{k.codes, k.exps, k.ld_codes, k.ld_exps};
        if (m) begin_matrix(m, ld);
        else
#pragma unroll
            for (int i = 0; i < C; ++i) codes[i] = ckpt_load8<G>(c, row, col[i], mask[i]);
    }
    __device__ __forceinline__ RowScalars begin_row(int64_t)
    {
        fetch(p.stream, p.ld_stream, p.stream_ckpt);
        const NormCommon& k = p.c;
        return RowScalars{k.post_norm ? p.rstd[row] : 1.0f, p.rstd[k.rows + row], gate_of_row<T>(k, row)};
    }
    __device__ __forceinline__ void begin_block() { fetch(p.block, p.ld_block, p.block_ckpt); }
    __device__ __forceinline__ void begin_dy() { begin_matrix(p.dy, p.ld_dy); }
    __device__ __forceinline__ void begin_du()
    {
        if (p.du) begin_matrix(p.du, p.ld_du);
    }
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

template <class T, int G, int C, bool ELEMENT>
__global__ void __launch_bounds__(C == 2 ? 512 : 1024) norm_backward_kernel(const NormBackParams p)
{
    pdl_enter();
    __shared__ __align__(16) float slots[2 * 3 * 32];
    SumSlots<3> sums(slots);
    int32_t col[C];
    uint32_t mask[C];
#pragma unroll
    for (int i = 0; i < C; ++i) {
        col[i] = first_col<G, C>(i);
        mask[i] = runs_below<G>(col[i], p.c.cols);
    }
    const Columns<T, G, C, false> cols{p.c, col, mask, 0};
    F8 sum_pre[C] = {}, sum_q[C] = {};
    float sum_scalar = 0.0f;
    for (int64_t row = blockIdx.x; row < p.c.rows; row += gridDim.x) {
        DirectLoader<T, G, C> in{p, col, mask, row};
        back_row<T, G, C, false, ELEMENT>(p, row, in, cols, sum_pre, sum_q, sum_scalar, sums);
    }
    store_sums<G, C>(p, col, mask, sum_pre, sum_q, sum_scalar);
}

constexpr int kSumThreads = 1024;

// Sums of the partial rows: a block takes 32 columns of one kind; its 32 warps
// each add a run of the partial rows in order, and the runs are added in
// order. Kind 0: d_pre; 1: Q, from which d_post and the gradient of a gate of
// columns follow; 2: the gradient of a scalar gate.
template <class T>
__global__ void __launch_bounds__(kSumThreads) norm_backward_sum_kernel(const NormBackParams p)
{
    pdl_enter();
    __shared__ float runs[kSumThreads / 32][32];
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
        const int per = (p.grid + kSumThreads / 32 - 1) / (kSumThreads / 32);
        const int end = min(p.grid, (warp + 1) * per);
#pragma unroll 8
        for (int b = warp * per; b < end; ++b) sum += src[b * step];
    }
    runs[warp][lane] = sum;
    __syncthreads();
    if (warp || !live) return;
    sum = 0.0f;
#pragma unroll
    for (int w = 0; w < kSumThreads / 32; ++w) sum += runs[w][lane];
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

// The queue form: two chunks per thread and 512 threads on an SM; wider rows
// leave no room for a row of copies ahead. They take four chunks in 1,024
// threads, whose five arrays of the row do not fit the registers: 1.8 to 4.6 KB
// of each thread's are spilled, and 5461 x 12288 from checkpoints takes 1,970 us,
// 2048 x 32768 1,240 (floor 99; 8192 x 8192 takes 130). A gate for each element,
// or one matrix beside one checkpoint, goes without the queue too (8192 x 4096:
// 265 and 120 us). (Two rows ahead of 16-bit elements:
// 8192 x 4096 from matrices 81 us instead of 77; 16384 x 8192 from checkpoints
// the same; issuing all of a row's copies during its exchange: 8192 x 4096 from
// checkpoints 74 us instead of 71.)
constexpr int64_t kQueueCols = kQueueThreads * 16;
// Shared memory of a block: the columns' parameters, the queues, the header.
template <class T, bool ODD>
size_t queue_bytes(int64_t threads)
{
    return threads * 2 * 64 + Queue<T, 2, 4, ODD>::bytes(threads) + Header<kHeaderRowsOf<T>>::size(threads);
}

template <class T, bool CKPT, bool ODD>
cudaError_t launch_queue(const NormBackParams& p, dim3 grid, unsigned threads, cudaStream_t s)
{
    auto kernel = norm_backward_queue_kernel<T, CKPT, ODD>;
    const cudaError_t e = cudaFuncSetAttribute((const void*)kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               (int)queue_bytes<T, ODD>(kQueueThreads));
    NormBackParams q = p;
    const int64_t saved = grid.x * (CKPT ? 1 : (int64_t)sizeof(T)), elements = grid.x * (int64_t)sizeof(T);
    q.step_stream = saved * (CKPT ? p.stream_ckpt.ld_codes : p.ld_stream);
    q.step_block = saved * (CKPT ? p.block_ckpt.ld_codes : p.ld_block);
    q.step_dy = elements * p.ld_dy;
    q.step_du = elements * p.ld_du;
    return e == cudaSuccess ? launch_kernel(kernel, grid, threads, queue_bytes<T, ODD>(threads), s, q) : e;
}

template <class T, int G, int C>
cudaError_t launch_direct(const NormBackParams& p, dim3 grid, unsigned threads, cudaStream_t s)
{
    return p.c.gate_cs && p.c.gate_rs ? launch_kernel(norm_backward_kernel<T, G, C, true>, grid, threads, 0, s, p)
                                      : launch_kernel(norm_backward_kernel<T, G, C, false>, grid, threads, 0, s, p);
}

template <class T>
cudaError_t launch(const NormBackParams& p, cudaStream_t s)
{
    const dim3 grid((unsigned)p.grid);
    const int64_t groups = (p.c.cols + 255) / 256;
    const unsigned by2 = (unsigned)((groups + 1) / 2) * 32, by4 = (unsigned)((groups + 3) / 4) * 32;
    // The queue takes rows of up to kQueueCols columns, a gate that is none or
    // varies along one axis, and two checkpoints or none.
    const bool element = p.c.gate_cs && p.c.gate_rs, mixed = !p.stream != !p.block;
    const bool vec = p.c.access == kAligned, odd = p.c.access == kOddPitch;
    cudaError_t e;
    if (p.c.cols > kQueueCols)
        e = vec ? launch_direct<T, kVector<T>, 4>(p, grid, by4, s) : launch_direct<T, 1, 4>(p, grid, by4, s);
    else if (element || mixed)
        e = vec ? launch_direct<T, kVector<T>, 2>(p, grid, by2, s) : launch_direct<T, 1, 2>(p, grid, by2, s);
    else if (vec)
        e = p.stream ? launch_queue<T, false, false>(p, grid, by2, s) : launch_queue<T, true, false>(p, grid, by2, s);
    else if (odd)
        e = p.stream ? launch_queue<T, false, true>(p, grid, by2, s) : launch_queue<T, true, true>(p, grid, by2, s);
    else
        e = launch_direct<T, 1, 2>(p, grid, by2, s);
    if (e != cudaSuccess) return e;
    if (!p.d_pre && !p.need_q && p.gate_kind != kGateScalar) return cudaSuccess;
    const dim3 sums((unsigned)((p.c.cols + 31) / 32), p.gate_kind == kGateScalar ? 3 : 2);
    return launch_kernel(norm_backward_sum_kernel<T>, sums, kSumThreads, 0, s, p);
}

}  // namespace

// One wave: the blocks that 512 threads of two chunks on each SM make up. The
// count is GB300's, not the device's answer: the order of the sums and the
// workspace then depend on the sizes alone.
int norm_backward_grid(int64_t rows, int64_t cols)
{
    constexpr int kSms = 152;
    const int64_t threads = (cols + 511) / 512 * 32;
    // (of few threads, as many as their shared memory leaves room for)
    const int64_t per_sm = threads >= 512 ? 1 : 512 / threads < 12 ? 512 / threads : 12;
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
