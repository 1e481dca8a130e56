// 8-bit activation checkpoints: [rows, cols] <-> int8 codes with one exponent
// byte for every 32 columns.
//
// Bound by HBM: 2 or 4 bytes per element in, 33/32 out (and back). One thread
// holds 8 columns; a warp covers 256 columns of one row, so a block's largest
// magnitude is two lane exchanges away and nothing is read twice.
#include "layers/layers_common.cuh"
#include "layers/layers_internal.h"

namespace ptoc {

namespace {

// Work unit u: 256 columns (one warp) of row u / units_per_row.
template <class T, bool V, bool RESTORE>
__global__ void __launch_bounds__(kBlock) ckpt8_kernel(const Ckpt8Params p)
{
    pdl_enter();
    const int64_t per_row = (p.cols + 255) / 256;
    const int64_t unit = (int64_t)blockIdx.x * (kBlock / 32) + (threadIdx.x >> 5);
    if (unit >= p.rows * per_row) return;
    const int64_t row = unit / per_row;
    const int64_t c = (unit - row * per_row) * 32 + (threadIdx.x & 31);
    const uint32_t mask = chunk_mask<V>(c, p.cols);
    const Ckpt k{p.ckpt.codes, p.ckpt.exps, p.ckpt.ld_codes, p.ckpt.ld_exps};
    T* x = (T*)p.x + row * p.ld;
    float v[8];
    if constexpr (RESTORE) {
        ckpt_load8<V>(k, row, c, mask, v);
        store8<T, V>(x, c, mask, v);
    } else {
        const Raw8<T> r = load8<T, V>(x, c, mask);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = r.at(j);
        ckpt_store8<V>(k, row, c, mask, v);
    }
}

template <class T, bool RESTORE>
cudaError_t launch(const Ckpt8Params& p, cudaStream_t s)
{
    const int64_t units = p.rows * ((p.cols + 255) / 256);
    const dim3 grid((unsigned)((units + kBlock / 32 - 1) / (kBlock / 32)));
    return p.vec ? launch_kernel(ckpt8_kernel<T, true, RESTORE>, grid, kBlock, 0, s, p)
                 : launch_kernel(ckpt8_kernel<T, false, RESTORE>, grid, kBlock, 0, s, p);
}

template <bool RESTORE>
cudaError_t dispatch(const Ckpt8Params& p, int dtype, cudaStream_t s)
{
    switch (dtype) {
    case PTOC_F32: return launch<float, RESTORE>(p, s);
    case PTOC_F16: return launch<__half, RESTORE>(p, s);
    default: return launch<__nv_bfloat16, RESTORE>(p, s);
    }
}

}  // namespace

cudaError_t launch_checkpoint8(const Ckpt8Params& p, int dtype, cudaStream_t s) { return dispatch<false>(p, dtype, s); }
cudaError_t launch_restore8(const Ckpt8Params& p, int dtype, cudaStream_t s) { return dispatch<true>(p, dtype, s); }

}  // namespace ptoc
