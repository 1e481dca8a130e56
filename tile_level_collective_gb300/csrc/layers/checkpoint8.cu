// 8-bit activation checkpoints: [rows, cols] <-> int8 codes with one exponent
// byte for every 32 columns.
//
// Bound by HBM: 2 or 4 bytes per element in, 33/32 out (and back). One thread
// holds 8 columns; a warp covers 256 columns of one row, so a block's largest
// magnitude is two lane exchanges away and nothing is read twice.
//
// Measured on GB300 (of 6.68 TB/s copied): 16384 x 8192 bf16 kept in 64 us (6.3
// TB/s), restored in 60 us (6.8 TB/s); with one 256-column unit per warp instead
// of four, and integer conversions, 105 and 147 us. At 8191 columns, element by
// element, 153 and 138 us: 8 loads or stores where an aligned row takes one.
#include "layers/layers_common.cuh"
#include "layers/layers_internal.h"

namespace ptoc {

namespace {

constexpr int kUnits = 4;            // work units whose loads a warp issues together

// Work unit u: 256 columns of row u / units_per_row, held by one warp. A block
// takes kUnits * 8 neighbouring units, its warps in turn.
template <class T, int G, bool RESTORE>
__global__ void __launch_bounds__(kBlock) ckpt8_kernel(const Ckpt8Params p)
{
    pdl_enter();
    const uint32_t per_row = (uint32_t)((p.cols + 255) / 256), units = (uint32_t)p.rows * per_row;
    const uint32_t unit0 = blockIdx.x * (kUnits * kBlock / 32) + (threadIdx.x >> 5);
    const Ckpt k{p.ckpt.codes, p.ckpt.exps, p.ckpt.ld_codes, p.ckpt.ld_exps};
    int64_t row[kUnits];
    int32_t col[kUnits];
    uint32_t mask[kUnits];
    Raw8<T, G> raw[kUnits];
    CkptRaw<G> codes[kUnits];
#pragma unroll
    for (int q = 0; q < kUnits; ++q) {
        const uint32_t unit = unit0 + q * (kBlock / 32);
        const uint32_t r = unit / per_row;
        row[q] = r;
        col[q] = (int32_t)((unit - r * per_row) * 256 + (threadIdx.x & 31) * G);
        mask[q] = unit < units ? runs_below<G>(col[q], p.cols) : 0u;
        if constexpr (RESTORE) codes[q] = ckpt_load8<G>(k, row[q], col[q], mask[q]);
        else raw[q] = load8<T, G>((const T*)p.x + row[q] * p.ld, col[q], mask[q]);
    }
#pragma unroll
    for (int q = 0; q < kUnits; ++q) {
        if (unit0 + q * (kBlock / 32) >= units) break;         // the whole warp
        if constexpr (RESTORE) store8<T, G>((T*)p.x + row[q] * p.ld, col[q], mask[q], ckpt_values<G>(codes[q], 1.0f));
        else ckpt_store8<G>(k, row[q], col[q], 0, mask[q], raw[q].expand());
    }
}

template <class T, bool RESTORE>
cudaError_t launch(const Ckpt8Params& p, cudaStream_t s)
{
    const int64_t units = p.rows * ((p.cols + 255) / 256);
    const int64_t per_block = kUnits * kBlock / 32;
    const dim3 grid((unsigned)((units + per_block - 1) / per_block));
    return p.vec ? launch_kernel(ckpt8_kernel<T, kVector<T>, RESTORE>, grid, kBlock, 0, s, p)
                 : launch_kernel(ckpt8_kernel<T, 1, RESTORE>, grid, kBlock, 0, s, p);
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
