// 8-bit activation checkpoints: [rows, cols] <-> int8 codes with one exponent
// byte for every 32 columns.
//
// Bound by HBM: 2 or 4 bytes per element in, 33/32 out (and back). One thread
// holds 8 columns; a warp covers 256 columns of one row, so a block's largest
// magnitude is two lane exchanges away and nothing is read twice.
//
// Measured on GB300 (of 6.79 TB/s copied): 16384 x 8192 bf16 kept in 64 us (6.3
// TB/s), restored in 60 us (6.8 TB/s); with one 256-column unit per warp instead
// of four, and integer conversions, 105 and 147 us. At 8191 columns 96 and 85 us:
// each run is put together from the two aligned words it lies across, with
// about 15 more instructions (element by element 154 and 138 us: 8 loads or
// stores where an aligned row takes one, and 8 exponents per chunk).
#include "layers/layers_common.cuh"
#include "layers/layers_internal.h"

namespace ptoc {

namespace {

// Work units whose loads a warp issues together: four, but fewer of rows of x
// that are read across words and take registers for both (16384 x 8191 with
// four, two and one: bf16 112, 96 and 100 us, binary32 184, 164 and 136).
template <class T, bool RESTORE, bool ACROSS>
constexpr int kUnitsOf = !ACROSS || RESTORE ? 4 : sizeof(T) == 2 ? 2 : 1;

// ---- rows of x at any address -----------------------------------------------------
// Runs of 16 bytes at any (element-aligned) address are moved as the aligned
// words that they lie across: `m` is the address modulo 16, the same for every
// run of a row.

// 16 bytes of lo and hi, from byte `m` (below 16) of lo on.
__device__ __forceinline__ void shift16(const uint32_t (&lo)[4], const uint32_t (&hi)[4], uint32_t m, uint32_t (&r)[4])
{
    uint32_t w[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
#pragma unroll
    for (int i = 0; i < 6; ++i) w[i] = m & 8 ? w[i + 2] : w[i];
#pragma unroll
    for (int i = 0; i < 5; ++i) w[i] = m & 4 ? w[i + 1] : w[i];
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = __funnelshift_r(w[i], w[i + 1], 8 * (m & 3));
}

// A chunk of a row of `cols`, loaded in two steps, so that the loads of several
// chunks are on their way together: the words that a run lies across, where
// both lie in the row, then what is left, by element.
template <class T, int G>
struct Across {
    static constexpr int S = (int)sizeof(T);
    uint4 lo[8 / G], hi[8 / G];

    static __device__ __forceinline__ bool words(uint32_t m, int32_t c, int32_t left)
    {
        return left >= G && (m == 0 || (c > 0 && left >= (32 - (int32_t)m) / S));
    }
    __device__ __forceinline__ void load(const T* row, int32_t col, int32_t cols)
    {
        const uint32_t m = (uint32_t)(uintptr_t)row & 15u;
#pragma unroll
        for (int q = 0; q < 8 / G; ++q) {
            const int32_t c = col + 32 * G * q;
            const uint4* at = (const uint4*)((const char*)(row + c) - m);
            const bool on = words(m, c, cols - c);
            lo[q] = hi[q] = make_uint4(0, 0, 0, 0);
            if (on) lo[q] = at[0];
            if (on && m) hi[q] = at[1];
        }
    }
    __device__ __forceinline__ Raw8<T, G> chunk(const T* row, int32_t col, int32_t cols) const
    {
        const uint32_t m = (uint32_t)(uintptr_t)row & 15u;
        Raw8<T, G> v;
#pragma unroll
        for (int q = 0; q < 8 / G; ++q) {
            const int32_t c = col + 32 * G * q, left = cols - c;
            uint32_t r[4];
            const uint32_t a[4] = {lo[q].x, lo[q].y, lo[q].z, lo[q].w}, b[4] = {hi[q].x, hi[q].y, hi[q].z, hi[q].w};
            shift16(a, b, m, r);
            if (!words(m, c, left) && left > 0) {
                using Word = std::conditional_t<S == 4, uint32_t, uint16_t>;
#pragma unroll
                for (int j = 0; j < G; ++j)
                    if (j < left) r[j * S / 4] |= (uint32_t)((const Word*)row)[c + j] << 8 * (j * S & 3);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) v.w[4 * q + i] = r[i];
        }
        return v;
    }
};

// The same for a store: a lane writes the aligned word that ends with the first
// bytes of its run and begins with the last ones of the lane before; what no
// lane covers so, at the ends of the warp and of the row, is written by element.
template <class T, int G>
__device__ __forceinline__ void store_across(T* row, int32_t col, int32_t cols, const Raw8<T, G>& v)
{
    constexpr int S = (int)sizeof(T);
    const uint32_t m = (uint32_t)(uintptr_t)row & 15u, lane = threadIdx.x & 31;
    const int32_t head = (16 - (int32_t)m) / S;             // elements of a run in the word before the boundary
#pragma unroll
    for (int q = 0; q < 8 / G; ++q) {
        const int32_t c = col + 32 * G * q, left = cols - c;
        const uint32_t own[4] = {v.w[4 * q], v.w[4 * q + 1], v.w[4 * q + 2], v.w[4 * q + 3]};
        uint32_t open = 0;                                  // elements that no word covers
        if (m == 0) {
            if (left >= G) *(uint4*)(row + c) = make_uint4(own[0], own[1], own[2], own[3]);
            else open = (1u << G) - 1;
        } else {
            uint32_t before[4], r[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) before[i] = __shfl_up_sync(0xffffffffu, own[i], 1);
            shift16(before, own, 16 - m, r);
            const uint32_t first = (1u << head) - 1, last = ((1u << G) - 1) & ~first;
            if (lane > 0 && left >= head) *(uint4*)((char*)(row + c) - m) = make_uint4(r[0], r[1], r[2], r[3]);
            else open = first;
            if (lane == 31 || left - G < head) open |= last;
        }
        if (left < G) open &= left > 0 ? (1u << left) - 1 : 0u;
        using Word = std::conditional_t<S == 4, uint32_t, uint16_t>;
#pragma unroll
        for (int j = 0; j < G; ++j)
            if (open >> j & 1) ((Word*)row)[c + j] = (Word)(own[j * S / 4] >> 8 * (j * S & 3));
    }
}

// The columns of the run that the end of the row cuts, if it lies in this chunk.
template <int G>
__device__ __forceinline__ int32_t cut_columns(int32_t col, uint32_t full, int32_t cols)
{
    const int32_t q = __popc(full);
    const int32_t left = cols - (col + 32 * G * q);
    return q < 8 / G && left > 0 ? left : 0;
}

// Which of the chunk's runs lie in the row as a whole.
template <int G>
__device__ __forceinline__ uint32_t whole_runs(int32_t col, int32_t cols)
{
    uint32_t m = 0;
#pragma unroll
    for (int q = 0; q < 8 / G; ++q) m |= cols - (col + 32 * G * q) >= G ? 1u << q : 0u;
    return m;
}

// Work unit u: 256 columns of row u / units_per_row, held by one warp. A block
// takes neighbouring units, its 8 warps in turn. ACROSS: rows of x at any
// address and of any length (the codes' rows are 8-byte aligned).
template <class T, int G, bool RESTORE, bool ACROSS>
__global__ void __launch_bounds__(kBlock) ckpt8_kernel(const Ckpt8Params p)
{
    constexpr int kUnits = kUnitsOf<T, RESTORE, ACROSS>;
    pdl_enter();
    const uint32_t per_row = (uint32_t)((p.cols + 255) / 256), units = (uint32_t)p.rows * per_row;
    const uint32_t unit0 = blockIdx.x * (kUnits * kBlock / 32) + (threadIdx.x >> 5);
    const Ckpt k{p.ckpt.codes, p.ckpt.exps, p.ckpt.ld_codes, p.ckpt.ld_exps};
    const int32_t cols = (int32_t)p.cols;
    int64_t row[kUnits];
    int32_t col[kUnits];
    uint32_t mask[kUnits];
    Raw8<T, G> raw[kUnits];
    Across<T, G> across[kUnits];
    CkptRaw<G> codes[kUnits];
#pragma unroll
    for (int q = 0; q < kUnits; ++q) {
        const uint32_t unit = unit0 + q * (kBlock / 32);
        const uint32_t r = unit / per_row;
        row[q] = r;
        col[q] = (int32_t)((unit - r * per_row) * 256 + (threadIdx.x & 31) * G);
        const int32_t end = unit < units ? cols : 0;
        mask[q] = ACROSS ? whole_runs<G>(col[q], end) : runs_below<G>(col[q], end);
        if constexpr (RESTORE) {
            codes[q] = ckpt_load8<G>(k, row[q], col[q], mask[q]);
            if constexpr (ACROSS) {
                const int32_t cut = cut_columns<G>(col[q], mask[q], end), n = __popc(mask[q]);
                if (cut > 0) {
                    const int32_t c = col[q] + 32 * G * n;
                    const uint8_t* from = (const uint8_t*)(k.codes + row[q] * k.ld_codes + c);
                    uint32_t w[2] = {};
#pragma unroll
                    for (int j = 0; j < G - 1; ++j)
                        if (j < cut) w[j / 4] |= (uint32_t)from[j] << 8 * (j & 3);
                    const uint32_t byte = k.exps[row[q] * k.ld_exps + (c >> 5)];
#pragma unroll
                    for (int g = 0; g < 8 / G; ++g)
                        if (g == n) {
                            codes[q].byte[g] = byte;
                            if constexpr (G == 8) codes[q].w[0] = w[0], codes[q].w[1] = w[1];
                            else codes[q].w[g] = w[0];
                        }
                }
            }
        } else if constexpr (ACROSS) {
            across[q].load((const T*)p.x + row[q] * p.ld, col[q], end);
        } else {
            raw[q] = load8<T, G>((const T*)p.x + row[q] * p.ld, col[q], mask[q]);
        }
    }
#pragma unroll
    for (int q = 0; q < kUnits; ++q) {
        if (unit0 + q * (kBlock / 32) >= units) break;         // the whole warp
        if constexpr (RESTORE) {
            T* to = (T*)p.x + row[q] * p.ld;
            const Raw8<T, G> v = round8<T, G>(ckpt_values<G>(codes[q], 1.0f));
            if constexpr (ACROSS) store_across<T, G>(to, col[q], cols, v);
            else store8<T, G>(to, col[q], mask[q], v);
        } else {
            if constexpr (ACROSS) raw[q] = across[q].chunk((const T*)p.x + row[q] * p.ld, col[q], cols);
            ckpt_store8<G>(k, row[q], col[q], 0, mask[q], raw[q].expand(),
                           ACROSS ? cut_columns<G>(col[q], mask[q], cols) : 0);
        }
    }
}

template <class T, bool RESTORE>
cudaError_t launch(const Ckpt8Params& p, cudaStream_t s)
{
    const int64_t units = p.rows * ((p.cols + 255) / 256);
    const int at_once = p.access == kOddPitch ? kUnitsOf<T, RESTORE, true> : kUnitsOf<T, RESTORE, false>;
    const int64_t per_block = at_once * kBlock / 32;
    const dim3 grid((unsigned)((units + per_block - 1) / per_block));
    switch (p.access) {
    case kAligned: return launch_kernel(ckpt8_kernel<T, kVector<T>, RESTORE, false>, grid, kBlock, 0, s, p);
    case kOddPitch: return launch_kernel(ckpt8_kernel<T, kVector<T>, RESTORE, true>, grid, kBlock, 0, s, p);
    default: return launch_kernel(ckpt8_kernel<T, 1, RESTORE, false>, grid, kBlock, 0, s, p);
    }
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
