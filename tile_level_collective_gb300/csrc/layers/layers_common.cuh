// Device pieces of the layer operators: rows in groups of 8 columns per
// thread, block-wide sums, and the 8-bit checkpoint code.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "reduce_impl.cuh"

namespace ptoc {

// ---- element conversions -------------------------------------------------------

template <class T>
__device__ __forceinline__ float to_f32(T v);
template <>
__device__ __forceinline__ float to_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ float to_f32<__half>(__half v) { return __half2float(v); }
template <>
__device__ __forceinline__ float to_f32<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }

template <class T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// ---- 8 columns per thread --------------------------------------------------------
// A row is cut into chunks of 8 columns; chunk c is held by one thread. With
// V (bases and pitches 16-byte aligned) a chunk is 8 neighbouring columns,
// moved as 16-byte words. Otherwise 32 neighbouring chunks, one per lane of a
// warp, cover their 256 columns with lane-contiguous elements (column 32 j +
// lane), so that element-wide accesses still coalesce. Either way 32 columns
// that share an exponent lie in one warp: 4 lanes (V), or element j of all
// lanes.

template <bool V>
__device__ __forceinline__ int64_t col_of(int64_t c, int j)
{
    if constexpr (V) return c * 8 + j;
    else return (c & ~(int64_t)31) * 8 + j * 32 + (c & 31);
}

// Elements of chunk c that lie below `cols`, as a bit mask.
template <bool V>
__device__ __forceinline__ uint32_t chunk_mask(int64_t c, int64_t cols)
{
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) m |= col_of<V>(c, j) < cols ? 1u << j : 0u;
    return m;
}

// The chunk's raw elements (zeros outside the mask); expanded later, so that
// several loads can be in flight in few registers.
template <class T>
struct Raw8 {
    Words<8 * sizeof(T) / 4> w;
    __device__ __forceinline__ float at(int j) const
    {
        if constexpr (sizeof(T) == 4) return __uint_as_float(w.w[j]);
        else {
            const uint32_t p = w.w[j >> 1];
            return to_f32(bitcast<T>((uint16_t)(j & 1 ? p >> 16 : p & 0xffffu)));
        }
    }
};

template <class T, bool V>
__device__ __forceinline__ Raw8<T> load8(const T* row, int64_t c, uint32_t mask)
{
    Raw8<T> r;
    if (V && mask == 0xffu) {
        const char* p = (const char*)(row + c * 8);
#pragma unroll
        for (int q = 0; q < (int)sizeof(T) / 2; ++q) {
            const Words<4> v = load_words<4>(p + 16 * q);
#pragma unroll
            for (int i = 0; i < 4; ++i) r.w.w[4 * q + i] = v.w[i];
        }
        return r;
    }
#pragma unroll
    for (int i = 0; i < (int)(8 * sizeof(T) / 4); ++i) r.w.w[i] = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j)
        if (mask >> j & 1) {
            const T v = row[col_of<V>(c, j)];
            if constexpr (sizeof(T) == 4) r.w.w[j] = __float_as_uint(v);
            else r.w.w[j >> 1] |= (uint32_t)bitcast<uint16_t>(v) << (j & 1 ? 16 : 0);
        }
    return r;
}

template <class T, bool V>
__device__ __forceinline__ void store8(T* row, int64_t c, uint32_t mask, const float* v)
{
    if (V && mask == 0xffu) {
        char* p = (char*)(row + c * 8);
#pragma unroll
        for (int q = 0; q < (int)sizeof(T) / 2; ++q) {
            Words<4> w;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if constexpr (sizeof(T) == 4) w.w[i] = __float_as_uint(v[4 * q + i]);
                else w.w[i] = (uint32_t)bitcast<uint16_t>(from_f32<T>(v[2 * i])) |
                              (uint32_t)bitcast<uint16_t>(from_f32<T>(v[2 * i + 1])) << 16;
            }
            store_words<4>(p + 16 * q, w);
        }
        return;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j)
        if (mask >> j & 1) row[col_of<V>(c, j)] = from_f32<T>(v[j]);
}

// Parameters (weights, gates): of the activations' type or binary32, read
// through the caches, every row again; one where null. Ordinary loads: a
// read-only load could be moved ahead of the wait for the previous kernel.
template <class T, bool V>
__device__ __forceinline__ void load_param8(const void* base, bool f32, int64_t c, uint32_t mask, float* v)
{
    if (!base) {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = 1.0f;
    } else if (V && mask == 0xffu) {
        if (f32 || sizeof(T) == 4) {
            const float4* p = (const float4*)((const float*)base + c * 8);
            const float4 a = p[0], b = p[1];
            v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
            v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
        } else {
            const uint4 a = *(const uint4*)((const T*)base + c * 8);
            const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                if constexpr (sizeof(T) == 2)
                    v[j] = to_f32(bitcast<T>((uint16_t)(j & 1 ? w[j >> 1] >> 16 : w[j >> 1] & 0xffffu)));
            }
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            v[j] = 0.0f;
            if (mask >> j & 1) {
                const int64_t k = col_of<V>(c, j);
                v[j] = f32 ? ((const float*)base)[k] : to_f32(((const T*)base)[k]);
            }
        }
    }
}

// ---- block-wide sums ---------------------------------------------------------------

// Sums of N values over the block, the same bits in every thread: lanes by a
// fixed exchange tree, then the warps' sums in order. `slot` is shared memory
// of N * 32 floats; two calls in a row need two slots (one barrier per call).
template <int N>
__device__ __forceinline__ void block_sum(float (&v)[N], float* slot)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
#pragma unroll
        for (int k = 0; k < N; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
    const int warps = (int)blockDim.x >> 5;
    if (warps == 1) return;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (lane == 0)
#pragma unroll
        for (int k = 0; k < N; ++k) slot[k * 32 + warp] = v[k];
    __syncthreads();
#pragma unroll
    for (int k = 0; k < N; ++k) {
        v[k] = lane < warps ? slot[k * 32 + lane] : 0.0f;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
    }
}

// ---- the 8-bit checkpoint code -------------------------------------------------------
// The shared exponent byte from the bits of the block's largest |x|: 127 is
// 1.984375 * 2^6, so the smallest e with |x| <= 127 * 2^e is the exponent of
// |x| minus 6, plus one when its mantissa is above that of 127 (0x7E0000):
// adding 0x1FFFF carries into the exponent field exactly then. 255 marks a
// block with an infinity or a NaN (their bits are the largest).
__device__ __forceinline__ uint32_t ckpt_exponent(uint32_t abs_bits)
{
    if (abs_bits >= 0x7f800000u) return 255u;
    const int e = (int)((abs_bits + 0x1ffffu) >> 23) - 6;
    return e > 0 ? (uint32_t)e : 0u;
}

// 2^(127 - byte), a normal number for every byte that ckpt_exponent gives (0
// to 249): the multiplication by it is exact but for results below 2^-126,
// which round to code 0 either way.
__device__ __forceinline__ float ckpt_inverse(uint32_t byte) { return __uint_as_float((254u - byte) << 23); }

// 2^(byte - 127); byte 0 is the subnormal 2^-127, byte 255 gives NaN (also
// times code 0).
__device__ __forceinline__ float ckpt_scale(uint32_t byte)
{
    return __uint_as_float(byte == 255u ? 0x7fc00000u : byte ? byte << 23 : 1u << 22);
}

__device__ __forceinline__ int ckpt_code(float x, float inverse) { return __float2int_rn(x * inverse); }

struct Ckpt {
    int8_t* codes;
    uint8_t* exps;
    int64_t ld_codes, ld_exps;
};

// Write chunk c (masked columns hold 0) of one row. Every lane of the warp
// takes part, also those whose mask is empty.
template <bool V>
__device__ __forceinline__ void ckpt_store8(const Ckpt& k, int64_t row, int64_t c, uint32_t mask, const float* v)
{
    int8_t* codes = k.codes + row * k.ld_codes;
    uint8_t* exps = k.exps + row * k.ld_exps;
    if constexpr (V) {
        uint32_t top = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) top = max(top, __float_as_uint(v[j]) & 0x7fffffffu);
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const uint32_t byte = ckpt_exponent(top);
        const float inv = byte == 255u ? 0.0f : ckpt_inverse(byte);
        int q[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) q[j] = byte == 255u ? 0 : ckpt_code(v[j], inv);
        if (mask == 0xffu) {
            Words<2> w;
#pragma unroll
            for (int i = 0; i < 2; ++i)
                w.w[i] = (uint32_t)(q[4 * i] & 255) | (uint32_t)(q[4 * i + 1] & 255) << 8 |
                         (uint32_t)(q[4 * i + 2] & 255) << 16 | (uint32_t)(q[4 * i + 3] & 255) << 24;
            store_words<2>((char*)(codes + c * 8), w);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (mask >> j & 1) codes[c * 8 + j] = (int8_t)q[j];
        }
        if (mask && (c & 3) == 0) exps[c >> 2] = (uint8_t)byte;
    } else {
        const int64_t block0 = (c & ~(int64_t)31) >> 2;      // 8 blocks of 32 columns per 32 chunks
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const uint32_t top = __reduce_max_sync(0xffffffffu, __float_as_uint(v[j]) & 0x7fffffffu);
            const uint32_t byte = ckpt_exponent(top);
            if (mask >> j & 1) {
                codes[col_of<false>(c, j)] = byte == 255u ? 0 : (int8_t)ckpt_code(v[j], ckpt_inverse(byte));
                if ((c & 31) == 0) exps[block0 + j] = (uint8_t)byte;
            }
        }
    }
}

// Read chunk c of one row (0 outside the mask).
template <bool V>
__device__ __forceinline__ void ckpt_load8(const Ckpt& k, int64_t row, int64_t c, uint32_t mask, float* v)
{
    const int8_t* codes = k.codes + row * k.ld_codes;
    const uint8_t* exps = k.exps + row * k.ld_exps;
    if (V && mask == 0xffu) {
        const Words<2> w = load_words<2>((const char*)(codes + c * 8));
        const float scale = ckpt_scale(exps[c >> 2]);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = (float)(int8_t)(w.w[j >> 2] >> (8 * (j & 3))) * scale;
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            v[j] = 0.0f;
            if (mask >> j & 1) {
                const int64_t col = col_of<V>(c, j);
                v[j] = (float)codes[col] * ckpt_scale(exps[col >> 5]);
            }
        }
    }
}

}  // namespace ptoc
