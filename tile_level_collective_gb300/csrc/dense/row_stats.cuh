// Mean and sum of squared deviations of a row that a block holds in registers.
#pragma once

#include "layers/layers_common.cuh"

namespace ptoc {

// A chunk's values where its mask allows, zeros elsewhere.
template <int G>
__device__ __forceinline__ F8 masked(const F8& f, uint32_t mask)
{
    if (mask == (1u << (8 / G)) - 1) return f;
    F8 r;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        float lo, hi;
        split(f.p[j], lo, hi);
        r.p[j] = pair(mask >> (2 * j / G) & 1 ? lo : 0.0f, mask >> ((2 * j + 1) / G) & 1 ? hi : 0.0f);
    }
    return r;
}

// The sum of a thread's values, or of their squares, in short chains.
template <int C, bool SQUARES>
__device__ __forceinline__ float sum_values(const F8 (&a)[C])
{
    Pair sum[2 * C];
#pragma unroll
    for (int i = 0; i < 2 * C; ++i) {
        const Pair u = a[i / 2].p[2 * (i & 1)], v = a[i / 2].p[2 * (i & 1) + 1];
        sum[i] = SQUARES ? fma2(u, u, mul2(v, v)) : add2(u, v);
    }
#pragma unroll
    for (int n = C; n > 0; n /= 2)
#pragma unroll
        for (int i = 0; i < n; ++i) sum[i] = add2(sum[i], sum[i + n]);
    return sum_of(sum[0]);
}

// R sums over the lanes, one beside the other.
template <int R>
__device__ __forceinline__ void lanes_sum(float (&v)[R])
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
#pragma unroll
        for (int r = 0; r < R; ++r) v[r] += __shfl_xor_sync(0xffffffffu, v[r], o);
}

// Each warp takes the mean of its own columns and the squared deviations from
// it; one exchange between the warps joins them:
//   d_w = mean_w - mean_0,  mean = mean_0 + sum(n_w d_w) / n
//   m2 = sum(m2_w) + sum(n_w d_w^2) - n (mean - mean_0)^2
// The last difference cannot lose more than a factor of n / n_0, the number of
// warps: what is subtracted is at most that times the sum of squares between
// the warps' means, which holds n_0 (mean_0 - mean)^2. n_w counts in whole warps (1,
// or a part of one), so that the sums do not leave binary32 before m2 does, which is
// above n_0 n_w / (n_0 + n_w) d_w^2 for every warp; counted in columns they would, by up
// to the number of warps. (n_w (mean_w - mean)^2 in a second turn over the slots:
// 16384 x 8192 bf16 182 us instead of 165.)
// C chunks of 256 columns to a warp, and no warp without columns; R rows at a
// time. The two slots are taken in turn, so one barrier per turn suffices.
template <int C, int R>
struct RowStats {
    static constexpr float kWarpCols = C * 256.0f;
    static constexpr int kSlots = 2 * R * 32;
    float2* slot;                       // [2][R][32]: mean and deviations of the warps
    float inv_mine, last, inv;          // 1 / columns of this warp; the last one's and 1 / all, in whole warps
    int warps, turn = 0;
    __device__ __forceinline__ RowStats(float2* s, int64_t cols) : slot(s), warps((int)(blockDim.x >> 5))
    {
        last = (float)(cols - (int64_t)(warps - 1) * C * 256);
        inv_mine = 1.0f / ((int)(threadIdx.x >> 5) == warps - 1 ? last : kWarpCols);
        last *= 1.0f / kWarpCols;
        inv = kWarpCols / (float)cols;
    }
    template <int G>
    __device__ __forceinline__ void of_rows(const F8 (&s)[R][C], const uint32_t (&mask)[C], float (&mean)[R],
                                            float (&m2)[R])
    {
#pragma unroll
        for (int r = 0; r < R; ++r) mean[r] = sum_values<C, false>(s[r]);
        lanes_sum<R>(mean);
#pragma unroll
        for (int r = 0; r < R; ++r) {
            mean[r] *= inv_mine;
            F8 d[C];
#pragma unroll
            for (int i = 0; i < C; ++i) {
#pragma unroll
                for (int j = 0; j < 4; ++j) d[i].p[j] = add2(s[r][i].p[j], both(-mean[r]));
                d[i] = masked<G>(d[i], mask[i]);
            }
            m2[r] = sum_values<C, true>(d);
        }
        lanes_sum<R>(m2);
        if (warps == 1) return;
        float2* at = slot + R * 32 * turn;
        turn ^= 1;
        if ((threadIdx.x & 31) == 0)
#pragma unroll
            for (int r = 0; r < R; ++r) at[32 * r + (threadIdx.x >> 5)] = make_float2(mean[r], m2[r]);
        __syncthreads();
        float mean0[R], shift[R], spread[R];
#pragma unroll
        for (int r = 0; r < R; ++r) mean0[r] = at[32 * r].x, shift[r] = spread[r] = m2[r] = 0.0f;
#pragma unroll 4
        for (int w = 0; w < warps; ++w) {
            const float n = w == warps - 1 ? last : 1.0f;
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const float2 v = at[32 * r + w];
                const float dw = v.x - mean0[r];
                shift[r] = fmaf(n, dw, shift[r]);
                spread[r] = fmaf(n * dw, dw, spread[r]);
                m2[r] += v.y;
            }
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const float delta = shift[r] * inv;
            mean[r] = mean0[r] + delta;
            m2[r] = fmaf(fmaxf(fmaf(-delta, shift[r], spread[r]), 0.0f), kWarpCols, m2[r]);
        }
    }
};

}  // namespace ptoc
