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

// ---- pairs of floats ------------------------------------------------------------------
// The kernels below issue several instructions per element and are close to
// the issue rate, so their arithmetic is written on pairs (one instruction for
// two binary32 operations, each rounded as usual).

using Pair = unsigned long long;

__device__ __forceinline__ Pair pair(float lo, float hi)
{
    Pair r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ Pair both(float v) { return pair(v, v); }
__device__ __forceinline__ void split(Pair p, float& lo, float& hi)
{
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(p));
}
__device__ __forceinline__ float sum_of(Pair p)
{
    float a, b;
    split(p, a, b);
    return a + b;
}
__device__ __forceinline__ Pair fma2(Pair a, Pair b, Pair c)
{
    Pair r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ Pair mul2(Pair a, Pair b)
{
    Pair r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ Pair add2(Pair a, Pair b)
{
    Pair r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// Eight columns in binary32.
struct F8 {
    Pair p[4];
};

// ---- 8 columns per thread ----------------------------------------------------------------
// A row is cut into groups of 256 columns, C neighbouring groups to a warp (so
// that the addresses of a lane's chunks differ by constants); of a group a lane
// holds a chunk of 8 columns as 8 / G runs of G neighbouring columns:
// G = 8, one 16-byte word of 16-bit elements; G = 4, two words of binary32;
// G = 1, element-wide accesses, for rows at any address and of any length. Run
// q of lane l starts at column 32 * G * q + G * l of the group, so that a warp
// always touches neighbouring words, and 32 columns that share an exponent lie
// in one run of neighbouring lanes. G > 1 needs 16-byte aligned bases and
// pitches and a multiple of G columns.

template <class T>
constexpr int kVector = 16 / (int)sizeof(T);

// The first column of this thread's chunk i of C. Signed, so that it is known
// not to wrap and its constant part stays one in 64-bit addresses.
template <int G, int C>
__device__ __forceinline__ int32_t first_col(int i)
{
    return (int32_t)(threadIdx.x >> 5) * (C * 256) + (int32_t)(threadIdx.x & 31) * G + i * 256;
}
// Which of the chunk's runs, from column `col` on, lie below `cols`.
template <int G>
__device__ __forceinline__ uint32_t runs_below(int32_t col, int64_t cols)
{
    uint32_t m = 0;
#pragma unroll
    for (int q = 0; q < 8 / G; ++q) m |= (int64_t)col + q * 32 * G < cols ? 1u << q : 0u;
    return m;
}

// A chunk as read: words of the type (G > 1), or one element per word.
template <class T, int G>
struct Raw8 {
    static constexpr int kWords = G == 1 ? 8 : 8 * (int)sizeof(T) / 4;
    uint32_t w[kWords];

    __device__ __forceinline__ F8 expand() const
    {
        F8 f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (sizeof(T) == 4) f.p[i] = pair(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
            else if constexpr (G == 1) f.p[i] = pair(widen(w[2 * i]), widen(w[2 * i + 1]));
            else f.p[i] = pair(widen(w[i] & 0xffffu), widen_high(w[i]));
        }
        return f;
    }
    static __device__ __forceinline__ float widen(uint32_t h)
    {
        if constexpr (std::is_same<T, __nv_bfloat16>::value) return __uint_as_float(h << 16);
        else return __half2float(bitcast<__half>((uint16_t)h));
    }
    static __device__ __forceinline__ float widen_high(uint32_t h)
    {
        if constexpr (std::is_same<T, __nv_bfloat16>::value) return __uint_as_float(h & 0xffff0000u);
        else return __half2float(bitcast<__half>((uint16_t)(h >> 16)));
    }
};

// `row` is the same for all threads, `col` this thread's first column; runs
// outside the mask give zeros. Ordinary loads: the wait for the previous
// kernel is a barrier for them, which it would not be for read-only loads.
template <class T, int G>
__device__ __forceinline__ Raw8<T, G> load8(const T* row, int32_t col, uint32_t mask)
{
    Raw8<T, G> r;
    const T* p = row + col;
    if constexpr (G == 1) {
        using Word = std::conditional_t<sizeof(T) == 4, uint32_t, uint16_t>;
        if (mask == 0xffu) {                // all but the row's last chunks
#pragma unroll
            for (int j = 0; j < 8; ++j) r.w[j] = *(const Word*)(p + 32 * j);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) r.w[j] = mask >> j & 1 ? *(const Word*)(p + 32 * j) : 0u;
        }
    } else {
#pragma unroll
        for (int q = 0; q < 8 / G; ++q) {
            uint4 v = make_uint4(0, 0, 0, 0);
            if (mask >> q & 1) v = *(const uint4*)(p + 32 * G * q);
            r.w[4 * q] = v.x, r.w[4 * q + 1] = v.y, r.w[4 * q + 2] = v.z, r.w[4 * q + 3] = v.w;
        }
    }
    return r;
}

// Two floats rounded to a word of two elements (the first in the low half).
template <class T>
__device__ __forceinline__ uint32_t pack2(Pair v)
{
    float lo, hi;
    split(v, lo, hi);
    if constexpr (std::is_same<T, __half>::value) return bitcast<uint32_t>(__floats2half2_rn(lo, hi));
    else return bitcast<uint32_t>(__floats2bfloat162_rn(lo, hi));
}

// The words that store8 writes.
template <class T, int G>
__device__ __forceinline__ Raw8<T, G> round8(const F8& v)
{
    Raw8<T, G> r;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (sizeof(T) == 4) {
            float lo, hi;
            split(v.p[i], lo, hi);
            r.w[2 * i] = __float_as_uint(lo), r.w[2 * i + 1] = __float_as_uint(hi);
        } else {
            const uint32_t w = pack2<T>(v.p[i]);
            if constexpr (G == 1) r.w[2 * i] = w & 0xffffu, r.w[2 * i + 1] = w >> 16;
            else r.w[i] = w;
        }
    }
    return r;
}

template <class T, int G>
__device__ __forceinline__ void store8(T* row, int32_t col, uint32_t mask, const Raw8<T, G>& r)
{
    T* p = row + col;
    if constexpr (G == 1) {
        using Word = std::conditional_t<sizeof(T) == 4, uint32_t, uint16_t>;
        if (mask == 0xffu) {
#pragma unroll
            for (int j = 0; j < 8; ++j) *(Word*)(p + 32 * j) = (Word)r.w[j];
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (mask >> j & 1) *(Word*)(p + 32 * j) = (Word)r.w[j];
        }
    } else {
#pragma unroll
        for (int q = 0; q < 8 / G; ++q)
            if (mask >> q & 1)
                *(uint4*)(p + 32 * G * q) = make_uint4(r.w[4 * q], r.w[4 * q + 1], r.w[4 * q + 2], r.w[4 * q + 3]);
    }
}

template <class T, int G>
__device__ __forceinline__ void store8(T* row, int32_t col, uint32_t mask, const F8& v)
{
    store8<T, G>(row, col, mask, round8<T, G>(v));
}

// Parameters (weights, gates) in the mapping of the activations: of their type
// or binary32; one where null, zero outside the mask.
template <class T, int G>
__device__ __forceinline__ F8 load_param8(const void* base, bool f32, int32_t col, uint32_t mask)
{
    F8 f;
    if (!base) {
#pragma unroll
        for (int i = 0; i < 4; ++i) f.p[i] = both(1.0f);
    } else if (f32 && sizeof(T) == 2) {
        float v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int q = j / G;
            v[j] = mask >> q & 1 ? ((const float*)base)[col + q * 32 * G + j % G] : 0.0f;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) f.p[i] = pair(v[2 * i], v[2 * i + 1]);
    } else {
        f = load8<T, G>((const T*)base, col, mask).expand();
    }
    return f;
}

// ---- block-wide sums ---------------------------------------------------------------

// Sums of N values over the block, the same bits in every thread: lanes by a
// fixed exchange tree, then the warps' sums by one. `begin` sums over the
// warp; what is done until `end` hides the wait for the other warps. The
// slots (2 * N * 32 floats, zeros at first) are taken in turn, so one barrier
// per sum suffices.
template <int N>
struct SumSlots {
    float* slot;
    int turn = 0;
    __device__ __forceinline__ explicit SumSlots(float* s) : slot(s)
    {
        for (int i = threadIdx.x; i < 2 * N * 32; i += blockDim.x) s[i] = 0.0f;
        __syncthreads();
    }
    __device__ __forceinline__ void begin(float (&v)[N])
    {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
#pragma unroll
            for (int k = 0; k < N; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
        if ((threadIdx.x & 31) == 0)
#pragma unroll
            for (int k = 0; k < N; ++k) slot[(turn * N + k) * 32 + (threadIdx.x >> 5)] = v[k];
    }
    __device__ __forceinline__ void end(float (&v)[N])
    {
        const float* s = slot + turn * N * 32;
        turn ^= 1;
        if (blockDim.x == 32) return;
        __syncthreads();
#pragma unroll
        for (int k = 0; k < N; ++k) {
            const float4* w = (const float4*)(s + 32 * k);
            auto four = [&](int i) {
                const float4 q = w[i];
                return (q.x + q.y) + (q.z + q.w);
            };
            v[k] = four(0) + four(1);
            if (blockDim.x > 256) v[k] += four(2) + four(3);
            if (blockDim.x > 512) v[k] += (four(4) + four(5)) + (four(6) + four(7));
        }
    }
    __device__ __forceinline__ void sum(float (&v)[N])
    {
        begin(v);
        end(v);
    }
};

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
constexpr float kCodeBias = 12582912.0f;

// Largest magnitude, or NaN if any is one.
__device__ __forceinline__ float max_abs(float a, float b)
{
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(fabsf(a)), "f"(fabsf(b)));
    return r;
}
__device__ __forceinline__ float max_abs(float a, float b, float c)
{
    float r;
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

struct Ckpt {
    int8_t* codes;
    uint8_t* exps;
    int64_t ld_codes, ld_exps;
};

// Write a chunk (zeros outside the mask) of one row: 256 * i columns after
// column `col0`. Every lane of the warp takes part, also those whose mask is
// empty. A run that the row's end cuts (G > 1) is not in the mask: the run
// after those that are has `cut` columns.
template <int G>
__device__ __forceinline__ void ckpt_store8(const Ckpt& k, int64_t row, int32_t col0, int i, uint32_t mask, const F8& f,
                                            int32_t cut = 0)
{
    int8_t* codes = k.codes + row * k.ld_codes + col0 + 256 * i;
    uint8_t* exps = k.exps + row * k.ld_exps + 8 * i;
    float v[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) split(f.p[i], v[2 * i], v[2 * i + 1]);
    if constexpr (G > 1) {
#pragma unroll
        for (int q = 0; q < 8 / G; ++q) {
            float top = max_abs(v[G * q], v[G * q + 1], v[G * q + 2]);
            if constexpr (G == 4) top = max_abs(top, v[G * q + 3]);
            else top = max_abs(max_abs(top, v[3], v[4]), max_abs(v[5], v[6], v[7]));
#pragma unroll
            for (int o = 1; o < 32 / G; o <<= 1) top = max_abs(top, __shfl_xor_sync(0xffffffffu, top, o));
            const uint32_t byte = ckpt_exponent(__float_as_uint(top));
            const Pair inv = both(ckpt_inverse(byte)), bias = both(kCodeBias);
            uint32_t w[G / 4];
#pragma unroll
            for (int n = 0; n < G / 4; ++n) {
                float c[4];
                split(fma2(f.p[(G * q + 4 * n) / 2], inv, bias), c[0], c[1]);
                split(fma2(f.p[(G * q + 4 * n) / 2 + 1], inv, bias), c[2], c[3]);
                w[n] = __byte_perm(__byte_perm(__float_as_uint(c[0]), __float_as_uint(c[1]), 0x0040),
                                   __byte_perm(__float_as_uint(c[2]), __float_as_uint(c[3]), 0x0040), 0x5410);
                if (byte == 255u) w[n] = 0u;
            }
            if (mask >> q & 1) {
                if constexpr (G == 8) *(uint2*)codes = make_uint2(w[0], w[G / 4 - 1]);
                else *(uint32_t*)(codes + 32 * G * q) = w[0];
                if ((threadIdx.x & (32 / G - 1)) == 0) exps[(col0 >> 5) + q * G] = (uint8_t)byte;
            } else if (cut > 0 && __popc(mask) == q) {
#pragma unroll
                for (int j = 0; j < G - 1; ++j)
                    if (j < cut) codes[32 * G * q + j] = (int8_t)(w[j / 4] >> 8 * (j & 3));
                if ((threadIdx.x & (32 / G - 1)) == 0) exps[(col0 >> 5) + q * G] = (uint8_t)byte;
            }
        }
    } else {
        // each exchange halves the elements whose largest a lane keeps, until the
        // lanes 4 j to 4 j + 3 share element j's: one exponent per lane, and the
        // lanes' inverses are handed back
        const uint32_t lane = threadIdx.x & 31;
        uint32_t top[8], code[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) top[j] = __float_as_uint(v[j]) & 0x7fffffffu;
#pragma unroll
        for (int n = 4; n > 0; n /= 2) {
            const bool upper = lane & (4 * n);
#pragma unroll
            for (int j = 0; j < n; ++j) {
                const uint32_t give = upper ? top[j] : top[j + n], keep = upper ? top[j + n] : top[j];
                top[j] = max(keep, __shfl_xor_sync(0xffffffffu, give, 4 * n));
            }
        }
        top[0] = max(top[0], __shfl_xor_sync(0xffffffffu, top[0], 2));
        top[0] = max(top[0], __shfl_xor_sync(0xffffffffu, top[0], 1));
        const uint32_t byte = ckpt_exponent(top[0]);
        const float inverse = byte == 255u ? 0.0f : ckpt_inverse(byte);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float inv = __shfl_sync(0xffffffffu, inverse, 4 * j);
            code[j] = inv == 0.0f ? 0u : __float_as_uint(__fmaf_rn(v[j], inv, kCodeBias));
        }
        if (mask == 0xffu) {
#pragma unroll
            for (int j = 0; j < 8; ++j) codes[32 * j] = (int8_t)code[j];
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (mask >> j & 1) codes[32 * j] = (int8_t)code[j];
        }
        const uint32_t any = __shfl_sync(0xffffffffu, mask, 0);        // a block exists where its first column does
        if ((lane & 3) == 0 && (any >> (lane >> 2) & 1))
            exps[((col0 - (int32_t)lane) >> 5) + (int32_t)(lane >> 2)] = (uint8_t)byte;
    }
}

// A chunk as read: code words (or single codes), and exponent bytes: one per
// run, or in lane j that of element j's block.
template <int G>
struct CkptRaw {
    uint32_t w[G == 1 ? 8 : 2];
    uint32_t byte[G == 4 ? 2 : 1];
};

template <int G>
__device__ __forceinline__ CkptRaw<G> ckpt_load8(const Ckpt& k, int64_t row, int32_t col, uint32_t mask)
{
    const int8_t* codes = k.codes + row * k.ld_codes + col;
    const uint8_t* exps = k.exps + row * k.ld_exps;
    CkptRaw<G> r;
    if constexpr (G == 8) {
        uint2 w = make_uint2(0, 0);
        if (mask) w = *(const uint2*)codes;
        r.w[0] = w.x, r.w[1] = w.y;
    } else if (G == 1 && mask == 0xffu) {
#pragma unroll
        for (int j = 0; j < 8; ++j) r.w[j] = *(const uint8_t*)(codes + 32 * j);
    } else {
#pragma unroll
        for (int j = 0; j < 8 / G; ++j) {
            r.w[j] = 0;
            if (mask >> j & 1)
                r.w[j] = G == 4 ? *(const uint32_t*)(codes + 128 * j) : *(const uint8_t*)(codes + 32 * j);
        }
    }
    if constexpr (G == 1) {
        const uint32_t any = __shfl_sync(0xffffffffu, mask, 0), lane = threadIdx.x & 31;
        r.byte[0] = 0;
        if (lane < 8 && (any >> lane & 1)) r.byte[0] = exps[((col - (int32_t)lane) >> 5) + (int32_t)lane];
    } else {
#pragma unroll
        for (int q = 0; q < 8 / G; ++q) {
            r.byte[q] = 0;
            if (mask >> q & 1) r.byte[q] = exps[(col + q * 32 * G) >> 5];
        }
    }
    return r;
}

// A code byte in the float 2^23 + 128 + code, without the slow integer
// conversion: with its sign bit flipped it is the lowest byte.
__device__ __forceinline__ float code_float(uint32_t flipped, int byte)
{
    return __uint_as_float(__byte_perm(flipped, 0x4b000000u, 0x7650 + byte));
}

// Code words as values, run q times scale[q] (G = 1: pair q of runs).
template <int G>
__device__ __forceinline__ F8 code_values(const uint32_t (&words)[G == 1 ? 8 : 2],
                                          const Pair (&scale)[G == 1 ? 4 : 8 / G])
{
    F8 f;
    const Pair bias = both(-8388736.0f);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (G == 1) {
            const Pair code = pair(code_float(words[2 * i] ^ 0x80u, 0), code_float(words[2 * i + 1] ^ 0x80u, 0));
            f.p[i] = mul2(add2(code, bias), scale[i]);
            continue;
        }
        const uint32_t w = words[i / 2] ^ 0x80808080u;
        f.p[i] = mul2(add2(pair(code_float(w, 2 * (i & 1)), code_float(w, 2 * (i & 1) + 1)), bias),
                      scale[G == 4 ? i / 2 : 0]);
    }
    return f;
}

// The chunk's values times `factor` (0 outside the mask, where codes are 0).
template <int G>
__device__ __forceinline__ F8 ckpt_values(const CkptRaw<G>& r, float factor)
{
    if constexpr (G == 1) {
        Pair scale[4];
        const float mine = ckpt_scale(r.byte[0]) * factor;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            scale[i] = pair(__shfl_sync(0xffffffffu, mine, 2 * i), __shfl_sync(0xffffffffu, mine, 2 * i + 1));
        return code_values<1>(r.w, scale);
    } else {
        Pair scale[8 / G];
#pragma unroll
        for (int q = 0; q < 8 / G; ++q) scale[q] = both(ckpt_scale(r.byte[q]) * factor);
        return code_values<G>(r.w, scale);
    }
}

// ---- queues of copies in shared memory -----------------------------------------------------
// Items (C chunks per thread of one row of one tensor) are copied ahead of
// their use, in the order of their use: K of them are always in flight or
// waiting. A warp copies and reads the bytes of its own columns only, in a
// part of the shared memory of its own. What lies past the row's end reads as
// zeros.
// Aligned rows (ODD = false): each lane copies and reads its own words, so
// that its own wait for the copy suffices; its words outside the mask are
// zeroed once and never copied to. Rows at any pitch (ODD; the base is
// 16-byte aligned): the lanes copy the aligned words that hold the warp's
// columns, one more than it has, and read elements where the row's address
// puts them; the lanes then wait for one another too. The word that holds the
// row's first element may begin in the row before.
template <class T, int C, int K, bool ODD>
struct Queue {
    static constexpr int G = ODD ? 1 : kVector<T>;
    static constexpr int W = (int)sizeof(T) / 2;             // words of 16 bytes per lane and chunk
    static constexpr uint32_t kChunk = (32 * W + (ODD ? 1 : 0)) * 16;       // bytes per warp
    static constexpr uint32_t kItem = C * kChunk, kWarp = K * kItem;
    static __host__ __device__ constexpr size_t bytes(size_t threads) { return threads / 32 * kWarp; }
    uint32_t at, first;                                      // the current slot; the first (of this lane, if !ODD)
    uint32_t lane;

    __device__ __forceinline__ Queue(void* smem, const uint32_t (&mask)[C])
    {
        lane = threadIdx.x & 31;
        first = at = (uint32_t)__cvta_generic_to_shared(smem) + (threadIdx.x >> 5) * kWarp + (ODD ? 0 : lane * 16);
        if constexpr (!ODD)
#pragma unroll
            for (int i = 0; i < C; ++i)
#pragma unroll
                for (int q = 0; q < W; ++q)
                    if (!(mask[i] >> q & 1))
                        for (int n = 0; n < K; ++n)
                            asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};"
                                         ::"r"(first + n * kItem + i * kChunk + q * 512), "r"(0) : "memory");
    }
    __device__ __forceinline__ uint32_t chunk_at(int i) const { return at + (uint32_t)i * kChunk; }
    static __device__ __forceinline__ void copy16(uint32_t dst, const void* src, uint32_t size)
    {
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(size) : "memory");
    }
    // This lane's word at byte `o` of the row's aligned words, which hold `total`
    // bytes up to the row's end; what lies past it is not read (a copy of no
    // bytes names the first word).
    static __device__ __forceinline__ void copy_part(uint32_t dst, const char* word0, int32_t o, int32_t total)
    {
        const int32_t bytes = min(max(total - o, 0), 16);
        copy16(dst, word0 + (bytes > 0 ? o : 0), (uint32_t)bytes);
    }
    // Start the copies of this warp's columns of a row of T.
    __device__ __forceinline__ void copy_row(const T* row, const int32_t (&col)[C], const uint32_t (&mask)[C],
                                             int64_t cols)
    {
#pragma unroll
        for (int i = 0; i < C; ++i) {
            if constexpr (ODD) {
                const char* word0 = (const char*)((uintptr_t)row & ~(uintptr_t)15);
                const int32_t total = (int32_t)((uintptr_t)row & 15) + (int32_t)cols * (int32_t)sizeof(T);
                const int32_t o = (col[i] - (int32_t)lane) * (int32_t)sizeof(T) + (int32_t)lane * 16;
#pragma unroll
                for (int q = 0; q <= W; ++q)
                    if (q < W || lane == 0) copy_part(chunk_at(i) + (lane + 32 * q) * 16, word0, o + 512 * q, total);
            } else {
#pragma unroll
                for (int q = 0; q < W; ++q)
                    if (mask[i] >> q & 1)
                        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;"
                                     ::"r"(chunk_at(i) + 512 * q), "l"(row + col[i] + 32 * G * q) : "memory");
            }
        }
    }
    // The same of a checkpoint's codes (aligned: one word of 8, or two of 4 bytes per lane).
    __device__ __forceinline__ void copy_codes(const int8_t* row, const int32_t (&col)[C], const uint32_t (&mask)[C],
                                               int64_t cols)
    {
#pragma unroll
        for (int i = 0; i < C; ++i) {
            if constexpr (ODD) {
                const char* word0 = (const char*)((uintptr_t)row & ~(uintptr_t)15);
                const int32_t total = (int32_t)((uintptr_t)row & 15) + (int32_t)cols;
                if (lane < 17)
                    copy_part(chunk_at(i) + lane * 16, word0, col[i] - (int32_t)lane + (int32_t)lane * 16, total);
            } else {
#pragma unroll
                for (int q = 0; q < W; ++q)
                    if (mask[i] >> q & 1)
                        asm volatile("cp.async.ca.shared.global [%0], [%1], %2;"
                                     ::"r"(chunk_at(i) + 512 * q), "l"(row + col[i] + 32 * G * q), "n"(ODD ? 8 : G)
                                     : "memory");
            }
        }
    }
    // The current slot is filled (or left as it is at the end): go on.
    __device__ __forceinline__ void next()
    {
        commit();
        at = at == first + kWarp - kItem ? first : at + kItem;
    }
    // Go to slot n (where the order of the items is known when compiling).
    __device__ __forceinline__ void go(int n) { at = first + (uint32_t)n * kItem; }
    __device__ __forceinline__ void commit() const { asm volatile("cp.async.commit_group;" ::: "memory"); }
    // Wait until the oldest item, which lies in the current slot, has landed.
    __device__ __forceinline__ void wait() const
    {
        asm volatile("cp.async.wait_group %0;" ::"n"(K - 1) : "memory");
        if constexpr (ODD) __syncwarp();
    }
    // The current slot has been read: it may be filled again.
    __device__ __forceinline__ void done() const
    {
        if constexpr (ODD) __syncwarp();
    }
    // Chunk i; `shift`: the row's address modulo 16.
    __device__ __forceinline__ Raw8<T, G> chunk(int i, uint32_t shift) const
    {
        Raw8<T, G> r;
        if constexpr (ODD) {
            const uint32_t from = chunk_at(i) + shift + lane * (uint32_t)sizeof(T);
            if constexpr (sizeof(T) == 4)
                asm volatile("ld.shared.u32 %0, [%8]; ld.shared.u32 %1, [%8 + 128];\n"
                             "ld.shared.u32 %2, [%8 + 256]; ld.shared.u32 %3, [%8 + 384];\n"
                             "ld.shared.u32 %4, [%8 + 512]; ld.shared.u32 %5, [%8 + 640];\n"
                             "ld.shared.u32 %6, [%8 + 768]; ld.shared.u32 %7, [%8 + 896];"
                             : "=&r"(r.w[0]), "=&r"(r.w[1]), "=&r"(r.w[2]), "=&r"(r.w[3]), "=&r"(r.w[4]), "=&r"(r.w[5]),
                               "=&r"(r.w[6]), "=&r"(r.w[7])
                             : "r"(from) : "memory");
            else
                asm volatile("{ .reg .u16 h<8>;\n"
                             "ld.shared.u16 h0, [%8]; ld.shared.u16 h1, [%8 + 64];\n"
                             "ld.shared.u16 h2, [%8 + 128]; ld.shared.u16 h3, [%8 + 192];\n"
                             "ld.shared.u16 h4, [%8 + 256]; ld.shared.u16 h5, [%8 + 320];\n"
                             "ld.shared.u16 h6, [%8 + 384]; ld.shared.u16 h7, [%8 + 448];\n"
                             "cvt.u32.u16 %0, h0; cvt.u32.u16 %1, h1; cvt.u32.u16 %2, h2; cvt.u32.u16 %3, h3;\n"
                             "cvt.u32.u16 %4, h4; cvt.u32.u16 %5, h5; cvt.u32.u16 %6, h6; cvt.u32.u16 %7, h7; }"
                             : "=&r"(r.w[0]), "=&r"(r.w[1]), "=&r"(r.w[2]), "=&r"(r.w[3]), "=&r"(r.w[4]), "=&r"(r.w[5]),
                               "=&r"(r.w[6]), "=&r"(r.w[7])
                             : "r"(from) : "memory");
        } else {
#pragma unroll
            for (int q = 0; q < W; ++q)
                asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                             : "=r"(r.w[4 * q]), "=r"(r.w[4 * q + 1]), "=r"(r.w[4 * q + 2]), "=r"(r.w[4 * q + 3])
                             : "r"(chunk_at(i) + 512 * q)
                             : "memory");
        }
        return r;
    }
    __device__ __forceinline__ void codes(int i, uint32_t shift, uint32_t (&w)[ODD ? 8 : 2]) const
    {
        if constexpr (ODD) {
            const uint32_t from = chunk_at(i) + shift + lane;
            asm volatile("ld.shared.u8 %0, [%8]; ld.shared.u8 %1, [%8 + 32]; ld.shared.u8 %2, [%8 + 64];\n"
                         "ld.shared.u8 %3, [%8 + 96]; ld.shared.u8 %4, [%8 + 128]; ld.shared.u8 %5, [%8 + 160];\n"
                         "ld.shared.u8 %6, [%8 + 192]; ld.shared.u8 %7, [%8 + 224];"
                         : "=&r"(w[0]), "=&r"(w[1]), "=&r"(w[2]), "=&r"(w[3]), "=&r"(w[4]), "=&r"(w[5]), "=&r"(w[6]),
                           "=&r"(w[7])
                         : "r"(from) : "memory");
        } else if constexpr (W == 1) {
            asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];"
                         : "=r"(w[0]), "=r"(w[1]) : "r"(chunk_at(i)) : "memory");
        } else {
#pragma unroll
            for (int q = 0; q < W; ++q)
                asm volatile("ld.shared.u32 %0, [%1];"
                             : "=r"(w[q]) : "r"(chunk_at(i) + 512 * q) : "memory");
        }
    }
};

}  // namespace ptoc
