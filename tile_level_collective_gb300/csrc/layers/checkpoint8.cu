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

constexpr int kUnits = 4;            // work units whose loads a warp issues together

// Work unit u: 256 columns of row u / units_per_row, held by one warp. A block
// takes kUnits * 8 neighbouring units, its warps in turn.
template <class T, bool V, bool RESTORE>
__global__ void __launch_bounds__(kBlock) ckpt8_kernel(const Ckpt8Params p)
{
    pdl_enter();
    const uint32_t per_row = (uint32_t)((p.cols + 255) / 256), units = (uint32_t)p.rows * per_row;
    const uint32_t unit0 = blockIdx.x * (kUnits * kBlock / 32) + (threadIdx.x >> 5);
    const Ckpt k{p.ckpt.codes, p.ckpt.exps, p.ckpt.ld_codes, p.ckpt.ld_exps};
    int64_t row[kUnits], c[kUnits];
    uint32_t mask[kUnits];
    Raw8<T> raw[kUnits];
    CkptRaw<V> codes[kUnits];
#pragma unroll
    for (int q = 0; q < kUnits; ++q) {
        const uint32_t unit = unit0 + q * (kBlock / 32);
        const uint32_t r = unit / per_row;
        row[q] = r;
        c[q] = (int64_t)(unit - r * per_row) * 32 + (threadIdx.x & 31);
        mask[q] = unit < units ? chunk_mask<V>(c[q], p.cols) : 0u;
        if constexpr (RESTORE) codes[q] = ckpt_load8<V>(k, row[q], c[q], mask[q]);
        else raw[q] = load8<T, V>((const T*)p.x + row[q] * p.ld, c[q], mask[q]);
    }
#pragma unroll
    for (int q = 0; q < kUnits; ++q) {
        if (unit0 + q * (kBlock / 32) >= units) break;         // the whole warp
        float v[8];
        if constexpr (RESTORE) {
            ckpt_values<V>(codes[q], 1.0f, v);
            store8<T, V>((T*)p.x + row[q] * p.ld, c[q], mask[q], v);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = raw[q].at(j);
            ckpt_store8<V>(k, row[q], c[q], mask[q], v);
        }
    }
}

template <class T, bool RESTORE>
cudaError_t launch(const Ckpt8Params& p, cudaStream_t s)
{
    const int64_t units = p.rows * ((p.cols + 255) / 256);
    const int64_t per_block = kUnits * kBlock / 32;
    const dim3 grid((unsigned)((units + per_block - 1) / per_block));
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
