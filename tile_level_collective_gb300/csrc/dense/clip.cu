// The global norm of a set of gradients and their scaling: one launch sums the
// squares, a second one takes the norm from the blocks' sums and scales. The
// gradients' addresses travel as kernel arguments, so nothing is copied to the
// device before the launch and a captured graph holds them; sets of more than
// kMaxItems take several launches of each kind.
//
// Bound by HBM: the set is read for the norm, and read and written for the
// scaling (from the end, where the norm's launch stopped: what is still in L2
// is not read again). A block takes neighbouring pieces of 8 KB, four at a time.
//
// Measured on GB300 (of 6.8 TB/s copied): 2^30 bf16 values, the norm alone 331 us
// (6.5 TB/s), out of place 992 us (6.5 TB/s); 2^29 f32 values 321 and 983 us; 2^24
// bf16 values 13 and 20 us, of which the launches and the blocks' sums are 8. 2^30
// zeros 412 and 1068 us (their squares are added a second time, scaled); 2^30 bf16
// values from an address that is no multiple of 16, element by element, 4350 and 8690.
#include <cmath>

#include "layers/layers_common.cuh"
#include "dense/dense_internal.h"

namespace ptoc {

namespace {

constexpr int kThreads = 512;
constexpr int kWords = 4;                   // 16-byte words of a thread in flight
constexpr int kBlocks = 2;                  // on an SM (three, with a few spilled registers: 2^30 bf16 values 1134 us, two 997)
constexpr int kGrid = kBlocks * 152;        // of a launch

// A gradient: `rows` rows of `cols` elements, cut into pieces. Packed ones are a single row.
struct Item {
    void *data, *out;
    int64_t ld, ld_out, cols, rows;
    int64_t first;                          // its first piece
    int32_t dtype;
    uint16_t words;                         // 1: rows of 16-byte words
    uint16_t rows_per;                      // rows of a piece
};

constexpr int kMaxItems = 400;              // 25.6 KB of the 32 KB of arguments that a launch takes
constexpr int kFewItems = 60;

template <int N>
struct ClipParams {
    Item item[N];
    int64_t pieces;
    double* partial;                        // one sum of squares per block of every launch
    float* result;
    float max_norm;
    int32_t count, first_block, blocks;     // of this launch; of all launches
    int32_t copies;                         // 1: some gradients have an output of their own
};

// Elements of a row in one piece (a word to a thread), and rows of a piece.
__host__ __device__ inline int64_t piece_cols(int dtype) { return kThreads * (dtype == PTOC_F32 ? 4 : 8); }
inline int64_t piece_rows(int64_t cols, int dtype)
{
    return cols >= piece_cols(dtype) ? 1 : piece_cols(dtype) / (cols > 0 ? cols : 1);
}
inline int64_t pieces_of(int64_t rows, int64_t cols, int dtype)
{
    const int64_t per = piece_rows(cols, dtype);
    return (rows + per - 1) / per * ((cols + piece_cols(dtype) - 1) / piece_cols(dtype));
}

// Rows [row, row + rows) and columns [col, col + cols) of a gradient.
struct Piece {
    int64_t row, col;
    uint32_t rows, cols;
};

// Pieces [n, n + count) of a packed gradient, or piece n of one with rows. (A
// division for every piece of a packed one: the norm of 2^24 bf16 values 39 us.)
__device__ __forceinline__ Piece piece_of(const Item& it, int64_t n, int64_t count)
{
    const int64_t pc = piece_cols(it.dtype);
    Piece s;
    if (it.rows == 1) {
        s.row = 0;
        s.col = n * pc;
        s.rows = 1;
        s.cols = (uint32_t)min(count * pc, it.cols - s.col);
        return s;
    }
    const int64_t across = (it.cols + pc - 1) / pc;
    const int64_t y = n / across, x = n - y * across;
    s.row = y * it.rows_per;
    s.col = x * pc;
    s.rows = (uint32_t)min((int64_t)it.rows_per, it.rows - s.row);
    s.cols = (uint32_t)min(pc, it.cols - s.col);
    return s;
}

__device__ __forceinline__ float read(const Item& it, int64_t at)
{
    if (it.dtype == PTOC_F32) return ((const float*)it.data)[at];
    if (it.dtype == PTOC_F16) return __half2float(((const __half*)it.data)[at]);
    return __bfloat162float(((const __nv_bfloat16*)it.data)[at]);
}

__device__ __forceinline__ void write(const Item& it, int64_t at, float v)
{
    if (it.dtype == PTOC_F32) ((float*)it.out)[at] = v;
    else if (it.dtype == PTOC_F16) ((__half*)it.out)[at] = __float2half_rn(v);
    else ((__nv_bfloat16*)it.out)[at] = __float2bfloat16_rn(v);
}

// f(place in the gradient, place in its output) for this thread's elements of a piece.
template <class F>
__device__ __forceinline__ void each_element(const Item& it, const Piece& s, F f)
{
    const uint32_t n = s.rows * s.cols;
    for (uint32_t i = threadIdx.x; i < n; i += kThreads) {
        const uint32_t r = i / s.cols, c = i - r * s.cols;
        f((s.row + r) * it.ld + s.col + c, (s.row + r) * it.ld_out + s.col + c);
    }
}

// This thread's words of a piece (at most kWords): f(q, word of the gradient,
// word of its output). A packed gradient's last elements are no word.
template <class F>
__device__ __forceinline__ void each_word(const Item& it, const Piece& s, F f)
{
    const uint32_t per = it.dtype == PTOC_F32 ? 4 : 8, across = s.cols / per, n = s.rows * across;
    const uint4 *data = (const uint4*)it.data;
    uint4* out = (uint4*)it.out;
    if (s.rows == 1) {
        const int64_t at = (s.row * it.ld + s.col) / per, to = (s.row * it.ld_out + s.col) / per;
        if (n == kThreads * kWords) {
#pragma unroll
            for (int q = 0; q < kWords; ++q) f(q, data + at + threadIdx.x + q * kThreads, out + to + threadIdx.x + q * kThreads);
        } else {
#pragma unroll
            for (int q = 0; q < kWords; ++q) {
                const uint32_t i = threadIdx.x + q * kThreads;
                if (i < n) f(q, data + at + i, out + to + i);
            }
        }
    } else {
#pragma unroll
        for (int q = 0; q < kWords; ++q) {
            const uint32_t i = threadIdx.x + q * kThreads;
            if (i >= n) continue;
            const uint32_t r = i / across, c = i - r * across;
            f(q, data + ((s.row + r) * it.ld + s.col) / per + c, out + ((s.row + r) * it.ld_out + s.col) / per + c);
        }
    }
}

// A word's elements as pairs of binary32.
template <class T>
constexpr int kPairs = sizeof(T) == 4 ? 2 : 4;

template <class T>
__device__ __forceinline__ void expand(const uint4& w, Pair (&f)[kPairs<T>])
{
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < kPairs<T>; ++i)
        if constexpr (sizeof(T) == 4) f[i] = pair(__uint_as_float(u[2 * i]), __uint_as_float(u[2 * i + 1]));
        else f[i] = pair(Raw8<T, 8>::widen(u[i] & 0xffffu), Raw8<T, 8>::widen_high(u[i]));
}

struct Words {
    uint4 w[kWords];
};

// The sum of squares of kWords words times `by`: words apart and then together,
// six additions at most, so off by at most 7 * 2^-24 of it with the squares'
// rounding.
template <class T>
__device__ __forceinline__ float scaled_squares(const Words& words, float by)
{
    Pair sum[kWords];
#pragma unroll
    for (int q = 0; q < kWords; ++q) {
        Pair f[kPairs<T>];
        expand<T>(words.w[q], f);
#pragma unroll
        for (int i = 0; i < kPairs<T>; ++i) {
            const Pair v = by == 1.0f ? f[i] : mul2(f[i], both(by));
            sum[q] = i == 0 ? mul2(v, v) : fma2(v, v, sum[q]);
        }
    }
    return sum_of(add2(add2(sum[0], sum[1]), add2(sum[2], sum[3])));
}

// The same where squares leave binary32's range (zeros come here too, and
// infinities and NaN, which stay): elements are scaled by a power of two, which
// is exact but for what is too small beside the rest.
template <class T>
__device__ __noinline__ double far_squares(Words words, bool small)
{
    constexpr double kUp = 0x1p100, kDown = 0x1p-70;
    return small ? (double)scaled_squares<T>(words, (float)kUp) * (1.0 / (kUp * kUp))
                 : (double)scaled_squares<T>(words, (float)kDown) * (1.0 / (kDown * kDown));
}

template <class T>
__device__ __forceinline__ double square_sum(const Words& words)
{
    const float s = scaled_squares<T>(words, 1.0f);
    if (s >= 1e-30f && s <= 1e30f) return (double)s;
    return far_squares<T>(words, s < 1e-30f);
}

template <class T>
__device__ __forceinline__ void scale_words(Words& words, Pair by)
{
#pragma unroll
    for (int q = 0; q < kWords; ++q) {
        Pair f[kPairs<T>];
        expand<T>(words.w[q], f);
        uint32_t u[4];
#pragma unroll
        for (int i = 0; i < kPairs<T>; ++i) {
            const Pair v = mul2(f[i], by);
            if constexpr (sizeof(T) == 4) {
                float lo, hi;
                split(v, lo, hi);
                u[2 * i] = __float_as_uint(lo), u[2 * i + 1] = __float_as_uint(hi);
            } else {
                u[i] = pack2<T>(v);
            }
        }
        words.w[q] = make_uint4(u[0], u[1], u[2], u[3]);
    }
}

// f(item, pieces) for the pieces of this block, up to kWords of one gradient at a
// time, from the first to the last or back.
template <int N, bool BACK, class F>
__device__ __forceinline__ void each_piece(const ClipParams<N>& p, F f)
{
    int64_t first = p.pieces * blockIdx.x / gridDim.x, last = p.pieces * (blockIdx.x + 1) / gridDim.x;
    if (first >= last) return;
    int lo = 0, hi = p.count - 1;                            // the item of the next piece
    for (const int64_t n = BACK ? last - 1 : first; lo < hi;) {
        const int mid = (lo + hi + 1) / 2;
        if (p.item[mid].first <= n) lo = mid;
        else hi = mid - 1;
    }
    while (first < last) {
        if (BACK)
            while (p.item[lo].first >= last) --lo;
        else
            while (lo + 1 < p.count && p.item[lo + 1].first <= first) ++lo;
        const Item& it = p.item[lo];
        const int64_t end = BACK || lo + 1 == p.count ? last : min(last, p.item[lo + 1].first);
        const int64_t begin = BACK ? max(first, it.first) : first;
        const int64_t count = it.rows == 1 ? min(end - begin, (int64_t)kWords) : 1;
        f(it, piece_of(it, (BACK ? end - count : begin) - it.first, count));
        if (BACK) last -= count;
        else first += count;
    }
}

// The elements of a packed gradient's piece that follow its last whole word.
__device__ __forceinline__ Piece rest_of(const Item& it, const Piece& s)
{
    const uint32_t per = it.dtype == PTOC_F32 ? 4 : 8, whole = s.cols / per * per;
    return Piece{s.row, s.col + whole, s.rows, s.cols - whole};
}

template <int N>
__global__ void __launch_bounds__(kThreads, kBlocks) clip_norm_kernel(const __grid_constant__ ClipParams<N> p)
{
    pdl_enter();
    __shared__ double sums[kThreads / 32];
    double sum = 0.0;
    auto elements = [&](const Item& it, const Piece& s) {
        each_element(it, s, [&](int64_t at, int64_t) {
            const double v = read(it, at);
            sum += v * v;
        });
    };
    each_piece<N, false>(p, [&](const Item& it, const Piece& s) {
        if (!it.words) {
            elements(it, s);
            return;
        }
        Words v = {};
        each_word(it, s, [&](int q, const uint4* from, uint4*) { v.w[q] = *from; });
        sum += it.dtype == PTOC_BF16  ? square_sum<__nv_bfloat16>(v)
               : it.dtype == PTOC_F16 ? square_sum<__half>(v) : square_sum<float>(v);
        elements(it, rest_of(it, s));
    });
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if ((threadIdx.x & 31) == 0) sums[threadIdx.x >> 5] = sum;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int w = 1; w < kThreads / 32; ++w) sum += sums[w];
        p.partial[p.first_block + blockIdx.x] = sum;
    }
}

// The norm, the same bits in every block: its threads share the blocks' sums,
// and theirs are added in order. (The last steps by one thread: binary64 takes 16
// cycles a warp.)
template <int N>
__device__ __forceinline__ void norm_of(const ClipParams<N>& p, double (&sums)[kThreads / 32], float& norm,
                                        float& scale)
{
    __shared__ float answer[2];
    double sum = 0.0;
    const int used = min((p.blocks + 31) & ~31, kThreads);
    if (threadIdx.x < used) {
        for (int b = threadIdx.x; b < p.blocks; b += kThreads) sum += p.partial[b];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if ((threadIdx.x & 31) == 0) sums[threadIdx.x >> 5] = sum;
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int w = 1; w < used / 32; ++w) sum += sums[w];
        const double root = sqrt(sum), ratio = (double)p.max_norm / (root + 1e-6);
        // (finite is what the caller reads: a root beyond binary32 is an infinite norm)
        answer[0] = (float)root;
        answer[1] = isfinite(answer[0]) && ratio < 1.0 ? (float)ratio : 1.0f;
    }
    __syncthreads();
    norm = answer[0];
    scale = answer[1];
}

template <int N>
__global__ void __launch_bounds__(kThreads, kBlocks) clip_scale_kernel(const __grid_constant__ ClipParams<N> p)
{
    pdl_enter();
    __shared__ double sums[kThreads / 32];
    float norm, scale;
    norm_of(p, sums, norm, scale);
    if (p.first_block == 0 && blockIdx.x == 0 && threadIdx.x == 0) {
        p.result[0] = norm;
        p.result[1] = scale;
    }
    if (scale == 1.0f && !p.copies) return;
    const Pair by = both(scale);
    auto elements = [&](const Item& it, const Piece& s) {
        each_element(it, s, [&](int64_t at, int64_t to) {
            if (scale != 1.0f) write(it, to, read(it, at) * scale);
            else if (it.dtype == PTOC_F32) ((uint32_t*)it.out)[to] = ((const uint32_t*)it.data)[at];
            else ((uint16_t*)it.out)[to] = ((const uint16_t*)it.data)[at];
        });
    };
    // what the norm's launch read last comes first: it may still be in L2
    each_piece<N, true>(p, [&](const Item& it, const Piece& s) {
        if (scale == 1.0f && it.out == it.data) return;
        if (!it.words) {
            elements(it, s);
            return;
        }
        Words v;
        each_word(it, s, [&](int q, const uint4* from, uint4*) { v.w[q] = *from; });
        if (scale != 1.0f) {
            if (it.dtype == PTOC_BF16) scale_words<__nv_bfloat16>(v, by);
            else if (it.dtype == PTOC_F16) scale_words<__half>(v, by);
            else scale_words<float>(v, by);
        }
        each_word(it, s, [&](int q, const uint4*, uint4* to) { *to = v.w[q]; });
        elements(it, rest_of(it, s));
    });
}

template <int N>
cudaError_t launch_group(const ptoc_gradient* grads, int count, int first_block, bool scale, int blocks,
                         float max_norm, float* result, double* partial, cudaStream_t s, int* used)
{
    ClipParams<N> p;
    p.pieces = 0;
    p.partial = partial;
    p.result = result;
    p.max_norm = max_norm;
    p.first_block = first_block;
    p.blocks = blocks;
    p.count = 0;
    p.copies = 0;
    for (int i = 0; i < count; ++i) {
        const ptoc_gradient& g = grads[i];
        Item it;
        it.data = g.data;
        it.out = g.out ? g.out : g.data;
        it.ld = g.ld;
        it.ld_out = g.out ? g.ld_out : g.ld;
        it.rows = g.rows;
        it.cols = g.cols;
        it.dtype = g.dtype;
        if (it.rows < 1 || it.cols < 1) continue;
        if ((it.ld == it.cols && it.ld_out == it.cols) || it.rows == 1) {
            it.cols *= it.rows;
            it.rows = 1;
        }
        const int64_t eb = g.dtype == PTOC_F32 ? 4 : 2;
        it.words = !(((uintptr_t)it.data | (uintptr_t)it.out |
                      (uintptr_t)(it.rows > 1 ? (it.ld | it.ld_out | it.cols) * eb : 0)) & 15u);
        it.rows_per = (uint16_t)piece_rows(it.cols, g.dtype);
        if (it.out != it.data) p.copies = 1;
        it.first = p.pieces;
        p.pieces += pieces_of(it.rows, it.cols, g.dtype);
        p.item[p.count++] = it;
    }
    const int grid = (int)(p.pieces < 1 ? 1 : p.pieces < kGrid ? p.pieces : kGrid);
    *used = grid;
    return scale ? launch_kernel(clip_scale_kernel<N>, dim3(grid), kThreads, 0, s, p)
                 : launch_kernel(clip_norm_kernel<N>, dim3(grid), kThreads, 0, s, p);
}

}  // namespace

size_t clip_workspace_bytes(int32_t count)
{
    const int launches = count <= 0 ? 1 : (count + kMaxItems - 1) / kMaxItems;
    return (size_t)launches * kGrid * sizeof(double);
}

cudaError_t launch_clip(const ptoc_gradient* grads, int32_t count, float max_norm, float* result, double* partial,
                        cudaStream_t s)
{
    int blocks = 0;
    for (int scale = 0; scale < 2; ++scale) {
        int at = 0, total = blocks;
        for (int i = 0; i == 0 || i < count; i += kMaxItems) {
            const int n = count - i < kMaxItems ? count - i : kMaxItems;
            int used = 0;
            const cudaError_t e =
                n <= kFewItems
                    ? launch_group<kFewItems>(grads + i, n, at, scale, total, max_norm, result, partial, s, &used)
                    : launch_group<kMaxItems>(grads + i, n, at, scale, total, max_norm, result, partial, s, &used);
            if (e != cudaSuccess) return e;
            at += used;
        }
        blocks = at;
    }
    return cudaSuccess;
}

}  // namespace ptoc
