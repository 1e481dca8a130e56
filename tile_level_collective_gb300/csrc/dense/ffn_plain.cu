// The gated feed-forward block and its backward pass on the CUDA cores, for
// operands at any address and pitch: every product is one kernel that reads
// both operands element by element. Where the tensor cores take h, dg and du as two
// numbers of the type (up to kPartsTokens tokens, or where the caller asks for it)
// they stay in binary32; elsewhere they are rounded to the type, as there.
#include "dense/ffn_act.cuh"
#include "dense/ffn_common.cuh"
#include "layers/layers_common.cuh"

namespace ptoc {

namespace {

constexpr int kTile = 64;                   // rows and columns of a block's result
constexpr int kStep = 16;                   // depth of a step
constexpr int kThreads = 256;               // 4 x 4 results each

// An operand: element (i, k) at base[i * si + k * sk].
struct Operand {
    const void* base;
    int64_t si, sk;
};

// result(m, n) = sum_k a(m, k) b(n, k), summed over up to two pairs of operands
// of the same depth: A's elements are of TA, B's and all others of T. MODE 0: stored;
// 1: a and b[0] give g, a and b[1] u, and the epilogue stores h (and pre); 2: dh, from
// which the epilogue stores dg, du and h. D: the elements of d, H: of MODE 2's h.
struct PlainParams {
    Operand a[2], b[2];
    int32_t pairs;
    int64_t m, n, k;
    void* d;
    int64_t ld_d;
    // MODE 1: d = h, pre may be null. MODE 2: pre is read, d = dg, d + plane = du
    void *pre, *h;
    int64_t ld_pre, inter, plane;
    int64_t tiles_n;
};

// A tile of an operand in shared memory, [k][i]: the direction in which
// addresses are neighbours goes along the threads.
template <class T>
__device__ __forceinline__ void load_tile(float (&to)[kStep][kTile + 4], const Operand& o, int64_t i0, int64_t k0,
                                          int64_t rows, int64_t depth)
{
#pragma unroll
    for (int e = threadIdx.x; e < kTile * kStep; e += kThreads) {
        const int i = o.sk == 1 ? e / kStep : e % kTile, k = o.sk == 1 ? e % kStep : e / kTile;
        float v = 0.0f;
        if (i0 + i < rows && k0 + k < depth) v = to_f32(((const T*)o.base)[(i0 + i) * o.si + (k0 + k) * o.sk]);
        to[k][i] = v;
    }
}

template <class TA, class T, class D, class H, int MODE, int ACT>
__global__ void __launch_bounds__(kThreads) ffn_plain_kernel(const PlainParams p)
{
    pdl_enter();
    constexpr int kB = MODE == 1 ? 2 : 1;
    __shared__ float as[kStep][kTile + 4], bs[kB][kStep][kTile + 4];
    const int64_t m0 = blockIdx.x / p.tiles_n * kTile, n0 = blockIdx.x % p.tiles_n * kTile;
    const int ty = threadIdx.x / 16 * 4, tx = threadIdx.x % 16 * 4;
    float acc[kB][4][4] = {};
    for (int pair = 0; pair < (MODE == 1 ? 1 : p.pairs); ++pair)
        for (int64_t k0 = 0; k0 < p.k; k0 += kStep) {
            load_tile<TA>(as, p.a[pair], m0, k0, p.m, p.k);
#pragma unroll
            for (int q = 0; q < kB; ++q) load_tile<T>(bs[q], p.b[MODE == 1 ? q : pair], n0, k0, p.n, p.k);
            __syncthreads();
#pragma unroll
            for (int k = 0; k < kStep; ++k)
#pragma unroll
                for (int q = 0; q < kB; ++q)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            acc[q][i][j] = fmaf(as[k][ty + i], bs[q][k][tx + j], acc[q][i][j]);
            __syncthreads();
        }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int64_t m = m0 + ty + i, n = n0 + tx + j;
            if (m >= p.m || n >= p.n) continue;
            D* d = (D*)p.d + m * p.ld_d + n;
            T* pre = (T*)p.pre + m * p.ld_pre + n;
            if constexpr (MODE == 0) {
                *d = from_f32<D>(acc[0][i][j]);
            } else if constexpr (MODE == 1) {
                const float g = acc[0][i][j], u = acc[kB - 1][i][j];
                *d = from_f32<D>(act_value<ACT>(g) * u);
                if (p.pre) pre[0] = from_f32<T>(g), pre[p.inter] = from_f32<T>(u);
            } else {
                const float dh = acc[0][i][j], u = to_f32(pre[p.inter]);
                const Act a = act_both<ACT>(to_f32(pre[0]));
                d[0] = from_f32<D>(dh * u * a.slope);
                d[p.plane] = from_f32<D>(dh * a.value);
                ((H*)p.h)[m * p.ld_d + n] = from_f32<H>(a.value * u);
            }
        }
}

template <class TA, class T, class D, class H, int MODE, int ACT>
cudaError_t run(PlainParams& p, cudaStream_t s)
{
    p.tiles_n = (p.n + kTile - 1) / kTile;
    const int64_t tiles = (p.m + kTile - 1) / kTile * p.tiles_n;
    return launch_kernel(ffn_plain_kernel<TA, T, D, H, MODE, ACT>, dim3((unsigned)tiles), kThreads, 0, s, p);
}

template <class T, class D, class H, int MODE>
cudaError_t run(PlainParams& p, int act, cudaStream_t s)
{
    return act == PTOC_ACT_SILU ? run<T, T, D, H, MODE, PTOC_ACT_SILU>(p, s)
                                : run<T, T, D, H, MODE, PTOC_ACT_GELU>(p, s);
}

// A result of one product.
template <class TA, class T, class TB = T>
cudaError_t product(Operand a, Operand b, int64_t m, int64_t n, int64_t k, void* d, int64_t ld, cudaStream_t s)
{
    PlainParams p = {};
    p.a[0] = a, p.b[0] = b, p.pairs = 1;
    p.m = m, p.n = n, p.k = k;
    p.d = d, p.ld_d = ld;
    return run<TA, TB, T, T, 0, 0>(p, s);
}

// W: the elements of h (its rows take as many bytes of the workspace as two parts).
template <class T, class W>
cudaError_t forward(const FfnParams& q, cudaStream_t s)
{
    const int64_t ip = padded_inter(q.inter);
    W* h = (W*)q.ws;
    PlainParams p = {};
    p.a[0] = Operand{q.x, q.ld_x, 1};
    p.b[0] = Operand{q.w_in, q.ld_in, 1};
    p.b[1] = Operand{(const T*)q.w_in + q.inter * q.ld_in, q.ld_in, 1};
    p.m = q.tokens, p.n = q.inter, p.k = q.hidden;
    p.d = h, p.ld_d = ip;
    p.pre = q.pre, p.ld_pre = q.ld_pre, p.inter = q.inter;
    const cudaError_t e = run<T, W, W, 1>(p, q.act, s);
    if (e != cudaSuccess) return e;
    return product<W, T>(Operand{h, ip, 1}, Operand{q.w_out, q.ld_out, 1}, q.tokens, q.hidden, q.inter, q.y, q.ld_y, s);
}

// W: the elements of dg and du; H: of h.
template <class T, class W, class H>
cudaError_t backward(const FfnBackParams& q, cudaStream_t s)
{
    // (a plane of two parts, or of one and its second one, has the bytes of binary32)
    constexpr bool kAll = sizeof(H) == 4;
    const BackLayout l = kAll ? parts_layout(q.tokens, q.inter) : back_layout(q.tokens, q.inter);
    const int64_t ip = l.ld, plane = kAll ? l.plane : l.plane * (int64_t)sizeof(T) / (int64_t)sizeof(W);
    W *dg = (W*)q.ws, *du = dg + plane;
    H* h = kAll ? (H*)(du + plane) : (H*)((T*)q.ws + l.h);
    PlainParams p = {};
    p.a[0] = Operand{q.dy, q.ld_dy, 1};
    p.b[0] = Operand{q.w_out, 1, q.ld_out};
    p.pairs = 1;
    p.m = q.tokens, p.n = q.inter, p.k = q.hidden;
    p.d = dg, p.ld_d = ip, p.plane = plane, p.h = h;
    p.pre = (void*)q.pre, p.ld_pre = q.ld_pre, p.inter = q.inter;
    cudaError_t e = run<T, W, H, 2>(p, q.act, s);
    const T* w_up = (const T*)q.w_in + q.inter * q.ld_in;
    if (e == cudaSuccess && q.dx) {
        PlainParams r = {};
        r.a[0] = Operand{dg, ip, 1}, r.a[1] = Operand{du, ip, 1};
        r.b[0] = Operand{q.w_in, 1, q.ld_in}, r.b[1] = Operand{w_up, 1, q.ld_in};
        r.pairs = 2;
        r.m = q.tokens, r.n = q.hidden, r.k = q.inter;
        r.d = q.dx, r.ld_d = q.ld_dx;
        e = run<W, T, T, T, 0, 0>(r, s);
    }
    const Operand x{q.x, 1, q.ld_x};
    if (e == cudaSuccess && q.d_in)
        e = product<W, T>(Operand{dg, 1, ip}, x, q.inter, q.hidden, q.tokens, q.d_in, q.ld_din, s);
    if (e == cudaSuccess && q.d_in)
        e = product<W, T>(Operand{du, 1, ip}, x, q.inter, q.hidden, q.tokens, (T*)q.d_in + q.inter * q.ld_din, q.ld_din,
                          s);
    if (e == cudaSuccess && q.d_out)
        e = product<T, T, H>(Operand{q.dy, 1, q.ld_dy}, Operand{h, 1, ip}, q.hidden, q.inter, q.tokens, q.d_out, q.ld_dout,
                          s);
    return e;
}

template <class T>
cudaError_t forward(const FfnParams& q, cudaStream_t s)
{
    return q.parts == 2 || q.tokens <= kPartsTokens ? forward<T, float>(q, s) : forward<T, T>(q, s);
}

template <class T>
cudaError_t backward(const FfnBackParams& q, cudaStream_t s)
{
    if (q.parts == 2) return backward<T, float, float>(q, s);
    return q.tokens <= kPartsTokens ? backward<T, float, T>(q, s) : backward<T, T, T>(q, s);
}

}  // namespace

cudaError_t launch_ffn_plain(const FfnParams& p, int dtype, cudaStream_t s)
{
    return dtype == PTOC_F16 ? forward<__half>(p, s) : forward<__nv_bfloat16>(p, s);
}

cudaError_t launch_ffn_backward_plain(const FfnBackParams& p, int dtype, cudaStream_t s)
{
    return dtype == PTOC_F16 ? backward<__half>(p, s) : backward<__nv_bfloat16>(p, s);
}

size_t ffn_workspace_bytes(int64_t tokens, int64_t, int64_t inter)
{
    const int64_t rows = tokens <= kFewTokens ? few_rows(tokens) * few_parts(tokens) : tokens;
    return (size_t)(rows * padded_inter(inter)) * 2;
}

size_t ffn_backward_workspace_bytes(int64_t tokens, int64_t, int64_t inter)
{
    return (size_t)back_layout(tokens, inter).elements * 2;
}

cudaError_t launch_ffn(const FfnParams& p, int dtype, cudaStream_t s)
{
    if (!p.vec) return launch_ffn_plain(p, dtype, s);
    return dtype == PTOC_F16 ? launch_ffn_tensor_f16(p, s) : launch_ffn_tensor_bf16(p, s);
}

cudaError_t launch_ffn_backward(const FfnBackParams& p, int dtype, cudaStream_t s)
{
    if (!p.vec) return launch_ffn_backward_plain(p, dtype, s);
    return dtype == PTOC_F16 ? launch_ffn_backward_tensor_f16(p, s) : launch_ffn_backward_tensor_bf16(p, s);
}

}  // namespace ptoc
