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
// A row is cut into chunks of 8 columns; chunk c is held by one thread. With V
// (bases and pitches 16-byte aligned, a multiple of 8 columns) a chunk is 8
// neighbouring columns, moved as 16-byte words. Otherwise 32 neighbouring
// chunks, one per lane of a warp, cover their 256 columns with lane-contiguous
// elements (column 32 j + lane), so that element-wide accesses still coalesce.
// Either way 32 columns that share an exponent lie in one warp: 4 lanes (V),
// or element j of all lanes. Loads and stores are predicated, not branched
// around, so that those of several chunks can be in flight together.

template <bool V>
__device__ __forceinline__ int64_t col_of(int64_t c, int j)
{
    if constexpr (V) return c * 8 + j;
    else return (c & ~(int64_t)31) * 8 + j * 32 + (c & 31);
}

// Elements of chunk c that lie below `cols`, as a bit mask (V: all or none).
template <bool V>
__device__ __forceinline__ uint32_t chunk_mask(int64_t c, int64_t cols)
{
    if constexpr (V) return c * 8 < cols ? 0xffu : 0u;
    const int64_t left = cols - col_of<V>(c, 0);        // element j is in if 32 j < left
    return left <= 0 ? 0u : left > 7 * 32 ? 0xffu : (1u << ((left + 31) / 32)) - 1u;
}

__device__ __forceinline__ Words<4> load16_if(const void* p, bool on)
{
    Words<4> r;
    asm volatile("{ .reg .pred p; setp.ne.u32 p, %5, 0;\n"
                 "mov.u32 %0, 0; mov.u32 %1, 0; mov.u32 %2, 0; mov.u32 %3, 0;\n"
                 "@p ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4]; }"
                 : "=&r"(r.w[0]), "=&r"(r.w[1]), "=&r"(r.w[2]), "=&r"(r.w[3]) : "l"(p), "r"((uint32_t)on) : "memory");
    return r;
}

__device__ __forceinline__ Words<2> load8_if(const void* p, bool on)
{
    Words<2> r;
    asm volatile("{ .reg .pred p; setp.ne.u32 p, %3, 0; mov.u32 %0, 0; mov.u32 %1, 0;\n"
                 "@p ld.global.L1::no_allocate.v2.u32 {%0, %1}, [%2]; }"
                 : "=&r"(r.w[0]), "=&r"(r.w[1]) : "l"(p), "r"((uint32_t)on) : "memory");
    return r;
}

__device__ __forceinline__ uint32_t load4_if(const void* p, bool on)
{
    uint32_t r;
    asm volatile("{ .reg .pred p; setp.ne.u32 p, %2, 0; mov.u32 %0, 0; @p ld.global.u32 %0, [%1]; }"
                 : "=&r"(r) : "l"(p), "r"((uint32_t)on) : "memory");
    return r;
}

__device__ __forceinline__ uint32_t load2_if(const void* p, bool on)
{
    uint32_t r;
    asm volatile("{ .reg .pred p; .reg .u16 h; setp.ne.u32 p, %2, 0; mov.u16 h, 0; @p ld.global.u16 h, [%1];\n"
                 "cvt.u32.u16 %0, h; }"
                 : "=&r"(r) : "l"(p), "r"((uint32_t)on) : "memory");
    return r;
}

__device__ __forceinline__ uint32_t load1_if(const void* p, bool on)
{
    uint32_t r;
    asm volatile("{ .reg .pred p; setp.ne.u32 p, %2, 0; mov.u32 %0, 0; @p ld.global.u8 %0, [%1]; }"
                 : "=&r"(r) : "l"(p), "r"((uint32_t)on) : "memory");
    return r;
}

// The chunk's raw elements (zeros outside the mask); expanded later, so that
// several loads can be in flight in few registers.
template <class T>
struct Raw8 {
    Words<8 * sizeof(T) / 4> w;
    __device__ __forceinline__ float at(int j) const
    {
        if constexpr (sizeof(T) == 4) return __uint_as_float(w.w[j]);
        else if constexpr (std::is_same<T, __nv_bfloat16>::value)
            return __uint_as_float(j & 1 ? w.w[j >> 1] & 0xffff0000u : w.w[j >> 1] << 16);
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
    if constexpr (V) {
        const char* p = (const char*)(row + c * 8);
#pragma unroll
        for (int q = 0; q < (int)sizeof(T) / 2; ++q) {
            const Words<4> v = load16_if(p + 16 * q, mask != 0);
#pragma unroll
            for (int i = 0; i < 4; ++i) r.w.w[4 * q + i] = v.w[i];
        }
    } else if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int j = 0; j < 8; ++j) r.w.w[j] = load4_if(row + col_of<V>(c, j), mask >> j & 1);
    } else {
        uint32_t h[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) h[j] = load2_if(row + col_of<V>(c, j), mask >> j & 1);
#pragma unroll
        for (int i = 0; i < 4; ++i) r.w.w[i] = h[2 * i] | h[2 * i + 1] << 16;
    }
    return r;
}

// Two floats rounded to a word of two elements (the first in the low half).
template <class T>
__device__ __forceinline__ uint32_t pack2(float lo, float hi)
{
    if constexpr (std::is_same<T, __half>::value) return bitcast<uint32_t>(__floats2half2_rn(lo, hi));
    else return bitcast<uint32_t>(__floats2bfloat162_rn(lo, hi));
}

template <class T, bool V>
__device__ __forceinline__ void store8(T* row, int64_t c, uint32_t mask, const float* v)
{
    if constexpr (V) {
        char* p = (char*)(row + c * 8);
#pragma unroll
        for (int q = 0; q < (int)sizeof(T) / 2; ++q) {
            Words<4> w;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if constexpr (sizeof(T) == 4) w.w[i] = __float_as_uint(v[4 * q + i]);
                else w.w[i] = pack2<T>(v[2 * i], v[2 * i + 1]);
            }
            asm volatile("{ .reg .pred p; setp.ne.u32 p, %5, 0; @p st.global.v4.u32 [%4], {%0, %1, %2, %3}; }"
                         ::"r"(w.w[0]), "r"(w.w[1]), "r"(w.w[2]), "r"(w.w[3]), "l"(p + 16 * q), "r"(mask)
                         : "memory");
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            T* p = row + col_of<V>(c, j);
            if constexpr (sizeof(T) == 4)
                asm volatile("{ .reg .pred p; setp.ne.u32 p, %2, 0; @p st.global.u32 [%1], %0; }"
                             ::"r"(__float_as_uint(v[j])), "l"(p), "r"(mask >> j & 1)
                             : "memory");
            else
                asm volatile("{ .reg .pred p; setp.ne.u32 p, %2, 0; @p st.global.u16 [%1], %0; }"
                             ::"h"(bitcast<uint16_t>(from_f32<T>(v[j]))), "l"(p), "r"(mask >> j & 1)
                             : "memory");
        }
    }
}

// Parameters (weights, gates): of the activations' type or binary32; one where
// null, zero outside the mask. Ordinary loads: a read-only load could be moved
// ahead of the wait for the previous kernel.
template <class T, bool V>
__device__ __forceinline__ void load_param8(const void* base, bool f32, int64_t c, uint32_t mask, float* v)
{
    if (!base) {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = 1.0f;
    } else if (f32) {
        const Raw8<float> r = load8<float, V>((const float*)base, c, mask);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = r.at(j);
    } else {
        const Raw8<T> r = load8<T, V>((const T*)base, c, mask);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = r.at(j);
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

// x / 2^e rounded to the nearest integer, ties to even, in the low byte of the
// result: x * 2^-e is exact and at most 127 in magnitude, and adding 1.5 * 2^23
// leaves no fraction bits, so the one rounding is that of the sum.
__device__ __forceinline__ uint32_t ckpt_code(float x, float inverse)
{
    return __float_as_uint(__fmaf_rn(x, inverse, 12582912.0f));
}

// Largest magnitude, or NaN if either is one.
__device__ __forceinline__ float max_abs(float a, float b)
{
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(fabsf(a)), "f"(fabsf(b)));
    return r;
}

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
        float top = max_abs(v[0], v[1]);
#pragma unroll
        for (int j = 2; j < 8; ++j) top = max_abs(top, v[j]);
        top = max_abs(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max_abs(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const uint32_t byte = ckpt_exponent(__float_as_uint(top));
        const float inv = ckpt_inverse(byte);
        uint32_t q[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) q[j] = ckpt_code(v[j], inv);
        uint32_t w[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            w[i] = __byte_perm(__byte_perm(q[4 * i], q[4 * i + 1], 0x0040),
                               __byte_perm(q[4 * i + 2], q[4 * i + 3], 0x0040), 0x5410);
            if (byte == 255u) w[i] = 0u;
        }
        asm volatile("{ .reg .pred p; setp.ne.u32 p, %3, 0; @p st.global.v2.u32 [%2], {%0, %1}; }"
                     ::"r"(w[0]), "r"(w[1]), "l"(codes + c * 8), "r"(mask)
                     : "memory");
        if (mask && (c & 3) == 0) exps[c >> 2] = (uint8_t)byte;
    } else {
        // lane j keeps the byte of element j's block and stores it
        const int64_t block0 = (c & ~(int64_t)31) >> 2;      // 8 blocks of 32 columns per 32 chunks
        uint32_t keep = 0, any = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const uint32_t top = __reduce_max_sync(0xffffffffu, __float_as_uint(v[j]) & 0x7fffffffu);
            const uint32_t byte = ckpt_exponent(top);
            const uint32_t code = byte == 255u ? 0u : ckpt_code(v[j], ckpt_inverse(byte));
            asm volatile("{ .reg .pred p; setp.ne.u32 p, %2, 0; @p st.global.u8 [%1], %0; }"
                         ::"r"(code), "l"(codes + col_of<false>(c, j)), "r"(mask >> j & 1)
                         : "memory");
            if ((c & 31) == j) keep = byte;
        }
        any = __shfl_sync(0xffffffffu, mask, 0);              // a block exists where its first column does
        if ((c & 31) < 8 && (any >> (c & 31) & 1)) exps[block0 + (c & 31)] = (uint8_t)keep;
    }
}

// Chunk c of one row as read: the codes and the exponent byte (V), or a code
// for each element and, in lane j, the byte of element j's block.
template <bool V>
struct CkptRaw {
    uint32_t w[V ? 2 : 8];
    uint32_t byte;
};

template <bool V>
__device__ __forceinline__ CkptRaw<V> ckpt_load8(const Ckpt& k, int64_t row, int64_t c, uint32_t mask)
{
    const int8_t* codes = k.codes + row * k.ld_codes;
    const uint8_t* exps = k.exps + row * k.ld_exps;
    CkptRaw<V> r;
    if constexpr (V) {
        const Words<2> w = load8_if(codes + c * 8, mask != 0);
        r.w[0] = w.w[0];
        r.w[1] = w.w[1];
        r.byte = load1_if(exps + (c >> 2), mask != 0);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) r.w[j] = load1_if(codes + col_of<V>(c, j), mask >> j & 1);
        const uint32_t any = __shfl_sync(0xffffffffu, mask, 0);
        const int lane = (int)(c & 31);
        r.byte = load1_if(exps + ((c & ~(int64_t)31) >> 2) + lane, lane < 8 && (any >> lane & 1));
    }
    return r;
}

// A code byte as a float, without the slow integer conversion: with its sign
// bit flipped it is the lowest byte of 2^23 + 128 + code.
__device__ __forceinline__ float code_value(uint32_t flipped, int byte)
{
    return __uint_as_float(__byte_perm(flipped, 0x4b000000u, 0x7650 + byte)) - 8388736.0f;
}

// The chunk's values times `factor` (0 outside the mask, which has codes 0).
template <bool V>
__device__ __forceinline__ void ckpt_values(const CkptRaw<V>& r, float factor, float* v)
{
    if constexpr (V) {
        const float scale = ckpt_scale(r.byte) * factor;
        const uint32_t w[2] = {r.w[0] ^ 0x80808080u, r.w[1] ^ 0x80808080u};
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = code_value(w[j >> 2], j & 3) * scale;
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float scale = ckpt_scale(__shfl_sync(0xffffffffu, r.byte, j)) * factor;
            v[j] = code_value(r.w[j] ^ 0x80u, 0) * scale;
        }
    }
}

// ---- a thread's queue of copies in shared memory ---------------------------------------
// Items (one chunk of C * 8 elements of one row of one tensor) are copied
// ahead of their use, in the order of their use: K of them are always in
// flight or waiting. A thread copies and reads its own bytes only, so nothing
// but its own wait for the copy is needed. Slots of 16 bytes per chunk word;
// W words of 16 bytes per chunk.
template <int C, int W, int K>
struct Queue {
    uint32_t base, stride, slot;
    static constexpr int kPerThread = C * W * 16;

    __device__ __forceinline__ Queue(void* smem)
    {
        stride = (uint32_t)blockDim.x * kPerThread;
        base = (uint32_t)__cvta_generic_to_shared(smem) + threadIdx.x * 16;
        slot = 0;
    }
    __device__ __forceinline__ uint32_t word(int i, int q) const
    {
        return base + slot * stride + (uint32_t)((i * W + q) * 16) * blockDim.x;
    }
    // Start the copy of `bytes` (16 or 8) into word (i, q) of the current slot.
    __device__ __forceinline__ void copy16(int i, int q, const void* src, bool on)
    {
        asm volatile("{ .reg .pred p; setp.ne.u32 p, %2, 0; @p cp.async.cg.shared.global [%0], [%1], 16; }"
                     ::"r"(word(i, q)), "l"(src), "r"((uint32_t)on)
                     : "memory");
    }
    __device__ __forceinline__ void copy8(int i, const void* src, bool on)
    {
        asm volatile("{ .reg .pred p; setp.ne.u32 p, %2, 0; @p cp.async.ca.shared.global [%0], [%1], 8; }"
                     ::"r"(word(i, 0)), "l"(src), "r"((uint32_t)on)
                     : "memory");
    }
    // The current slot is filled (or left empty at the end): go on.
    __device__ __forceinline__ void next()
    {
        asm volatile("cp.async.commit_group;" ::: "memory");
        slot = slot + 1 == K ? 0 : slot + 1;
    }
    // Wait until the oldest item, which lies in the current slot, has landed.
    __device__ __forceinline__ void wait() const { asm volatile("cp.async.wait_group %0;" ::"n"(K - 1) : "memory"); }
    __device__ __forceinline__ Words<4> read(int i, int q) const
    {
        Words<4> r;
        asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(r.w[0]), "=r"(r.w[1]), "=r"(r.w[2]), "=r"(r.w[3]) : "r"(word(i, q)) : "memory");
        return r;
    }
    // The words of chunk i in every slot read as zeros: for a chunk past the row's end.
    __device__ __forceinline__ void clear(int i)
    {
        for (slot = 0; slot < K; ++slot)
#pragma unroll
            for (int q = 0; q < W; ++q)
                asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(word(i, q)), "r"(0) : "memory");
        slot = 0;
    }
    template <class T>
    __device__ __forceinline__ Raw8<T> chunk(int i) const
    {
        Raw8<T> r;
#pragma unroll
        for (int q = 0; q < W; ++q) {
            const Words<4> v = read(i, q);
#pragma unroll
            for (int k = 0; k < 4; ++k) r.w.w[4 * q + k] = v.w[k];
        }
        return r;
    }
    // Start the copies of a row's chunks of this thread: elements of T.
    template <class T>
    __device__ __forceinline__ void copy_row(const T* row, const uint32_t (&mask)[C])
    {
#pragma unroll
        for (int i = 0; i < C; ++i)
#pragma unroll
            for (int q = 0; q < W; ++q)
                copy16(i, q, (const char*)(row + ((int64_t)i * blockDim.x + threadIdx.x) * 8) + 16 * q, mask[i] != 0);
    }
};

}  // namespace ptoc
