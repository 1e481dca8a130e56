// The gated feed-forward block for a few tokens (up to kFewTokens): launches of
// one kernel that streams weights through shared memory into tcgen05.mma, two in
// the forward pass and two for the backward pass' dg, du, h and dx.
//
//   kIn       64 gate and the matching 64 up rows x hidden        h (and pre)
//   kOut      128 rows of w_out x inter                           y
//   kBackIn   128 columns of w_out x hidden                       dg, du and h
//   kBackX    128 columns of w_in x the gate's, then the up inter dx
//
// Bound by HBM: 3 * inter * hidden weights, read once. The rows of an mma are 128
// rows (or, read along the other direction, columns) of weights, its columns the
// call's tokens, padded to NT = 8, 16, 32, 64 or 128. The depth of a tile is split over a cluster of up to 8 blocks, so that
// small blocks and the second product, whose tiles are few and deep, fill the
// GPU too; two blocks share an SM, so that one's start and end lie within the
// other's stream. The blocks of a cluster leave their partial sums in shared
// memory and add them there, each a part of the tile, in the order of the depth:
// no partial sum passes through HBM, and the order does not depend on scheduling.
//
// Up to 64 tokens the second product has 2 NT columns: h as two numbers of the
// type (split_parts.cuh), whose sums are added at the end; with more, one. It is launched while the
// first one runs, and its first weights are on their way before it waits for h.
//
// Measured on GB300 (bf16, 4096 x 12288, of 6.8 TB/s copied): 1 token 52 us forward
// (5.8 TB/s; under ncu the products take 35 and 22 us), dg, du, h and dx 51 us; 64
// tokens 62 and 61 us; 128 tokens 69 and 67. What a call costs beside its stream
// of weights: the first copies (2 us), the partial sums' exchange (2 us), the
// launches. The tensor cores are 4 % busy at 1 token and 15 to 25 % at 64.
#pragma once

#include "dense/ffn_act.cuh"
#include "dense/ffn_common.cuh"
#include "layers/layers_common.cuh"
#include "layers/split_parts.cuh"
#include "layers/tensor_core.cuh"

namespace ptoc {

namespace {

namespace few {

constexpr int kDepth = 64;
constexpr int kRows = 128;                  // of a tile of weights
constexpr int kThreads = 256;               // warp 0 copies, warp 1 multiplies, warps 4 to 7 drain; all add
constexpr int kMaxStages = 6;
constexpr int kMaxSplit = 8;
constexpr int kSlots = 2 * 152;             // blocks at a time

enum Form : int { kIn = 0, kOut = 1, kBackIn = 2, kBackX = 3 };
// The second product of either pass: its tokens' rows are the first one's results.
template <int FORM>
constexpr bool kSecond = FORM == kOut || FORM == kBackX;

struct Params {
    CUtensorMap w, x;                       // weights; tokens' rows (second products: both parts)
    void *out, *pre;                        // kIn: h's parts, [kParts * NT, inter]; kBackIn: dg's; kOut: y; kBackX: dx
    void* h;                                // kBackIn: h, [tokens, inter]
    int64_t ld_out, ld_pre, inter;
    int64_t plane;                          // kBackIn: from dg's parts to du's
    int32_t tokens, rows;                   // rows of the result's other side (inter or hidden)
    int32_t depth, plane_depth;             // stages of a tile, and of one plane of the weights
    int32_t split;                          // blocks of a cluster
    uint64_t wait_ns;
};

struct Shared {
    uint64_t full[kMaxStages], empty[kMaxStages], done;
    uint32_t tmem;
    int32_t fault;
    uint32_t armed;
};

constexpr uint32_t kHead = 1024;
constexpr uint32_t kSharedMost = 113 * 1024;         // two blocks to an SM
// Numbers that stand for an element of h, dg or du. With two, 128 tokens would have 48 KB
// to a stage, 32 of them tokens.
template <int NT>
constexpr int kParts = NT <= kPartsTokens ? 2 : 1;
template <int FORM, int NT>
constexpr int kColumns = kSecond<FORM> ? kParts<NT> * NT : NT < 16 ? 16 : NT;
template <int FORM, int NT>
constexpr uint32_t kStageBytes = (kRows + kColumns<FORM, NT>) * kDepth * 2;
template <int FORM, int NT>
constexpr int kStages = (int)((kSharedMost - kHead - 1024) / kStageBytes<FORM, NT>) < kMaxStages
                            ? (int)((kSharedMost - kHead - 1024) / kStageBytes<FORM, NT>)
                            : kMaxStages;
template <int FORM, int NT>
constexpr uint32_t kSharedBytes = kHead + 1024 + kStages<FORM, NT> * kStageBytes<FORM, NT>;

__device__ __forceinline__ void mma(uint32_t d, uint64_t a, uint64_t b, uint32_t kind, uint32_t accumulate)
{
    asm volatile("{ .reg .pred p; setp.ne.u32 p, %4, 0;\n"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p; }"
                 ::"r"(d), "l"(a), "l"(b), "r"(kind), "r"(accumulate)
                 : "memory");
}

__device__ __forceinline__ void commit(uint64_t* bar)
{
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar))
                 : "memory");
}

__device__ __forceinline__ bool wait(Shared& sh, uint64_t* bar, uint32_t parity, uint64_t bound_ns)
{
    if (bounded_wait(smem_u32(bar), parity, bound_ns, &sh.fault)) return true;
    if (atomicExch(&sh.fault, 1) == 0) atomicAdd(&g_stage_faults, 1u);
    return false;
}

__device__ __forceinline__ float remote_float(uint32_t addr)
{
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}

// Tokens that a thread adds the partial sums of at a time: as many loads on their way.
constexpr int kAtOnce = 4;

// The sums of `count` elements, `pitch` bytes apart, over the cluster's blocks, in their order.
__device__ __forceinline__ void sums_of_blocks(uint32_t addr, uint32_t pitch, int count, int split,
                                               float (&sum)[kAtOnce])
{
    float v[kMaxSplit][kAtOnce];
#pragma unroll
    for (int s = 0; s < kMaxSplit; ++s)
        if (s < split) {
            const uint32_t at = in_block(addr, s);
#pragma unroll
            for (int j = 0; j < kAtOnce; ++j) v[s][j] = j < count ? remote_float(at + j * pitch) : 0.0f;
        }
#pragma unroll
    for (int j = 0; j < kAtOnce; ++j) {
        sum[j] = v[0][j];
#pragma unroll
        for (int s = 1; s < kMaxSplit; ++s)
            if (s < split) sum[j] += v[s][j];
    }
}

template <class T, int FORM, int ACT, int NT>
__global__ void __launch_bounds__(kThreads, 2) ffn_few_kernel(const __grid_constant__ Params p)
{
    extern __shared__ unsigned char raw[];
    Shared& sh = *(Shared*)raw;
    constexpr int kCols = kColumns<FORM, NT>;
    constexpr uint32_t kRing = kStages<FORM, NT>, kStage = kStageBytes<FORM, NT>, kWeightBytes = kRows * kDepth * 2;
    constexpr uint32_t kTmem = kCols < 32 ? 32 : kCols;
    constexpr uint32_t kType = std::is_same<T, __half>::value ? 0u : 1u;
    constexpr bool kByRows = FORM == kBackIn || FORM == kBackX;   // the weights' rows run along the depth
    constexpr uint32_t kKind = 1u << 4 | kType << 7 | kType << 10 | (uint32_t)kByRows << 15 |
                               (uint32_t)(kCols >> 3) << 17 | (kRows >> 4) << 24;
    const uint32_t ring = (smem_u32(raw) + kHead + 1023u) & ~1023u;
    const int lane = threadIdx.x & 31, warp = uniform_warp();
    const int rank = (int)cluster_rank(), tile = (int)blockIdx.x / p.split;
    const int first = (int)((int64_t)p.depth * rank / p.split), last = (int)((int64_t)p.depth * (rank + 1) / p.split);

    // A second product reads its weights before it waits: the launch before it
    // in the stream is the first product, which waited for everything before. (The
    // header forbids other threads to put a launch that writes weights between the
    // two: one that releases its dependents early would not be waited for.) A
    // warp of its own starts these copies while another one allocates.
    auto weights = [&](int x, uint32_t slot) {
        const uint32_t dst = ring + slot * kStage;
        bar_expect(&sh.full[slot], kStage);
        if constexpr (FORM == kIn) {
            copy_box(dst, &p.w, x * kDepth, tile * (kRows / 2), 0, &sh.full[slot]);
            copy_box(dst + kWeightBytes / 2, &p.w, x * kDepth, tile * (kRows / 2), 1, &sh.full[slot]);
        } else if constexpr (FORM == kOut) {
            copy_box(dst, &p.w, x * kDepth, tile * kRows, 0, &sh.full[slot]);
        } else {
            const int plane = FORM == kBackX && x >= p.plane_depth, y = (x - plane * p.plane_depth) * kDepth;
            copy_box(dst, &p.w, tile * kRows, y, plane, &sh.full[slot]);
            copy_box(dst + kWeightBytes / 2, &p.w, tile * kRows + 64, y, plane, &sh.full[slot]);
        }
    };
    auto tokens = [&](int x, uint32_t slot) {
        const int plane = FORM == kBackX && x >= p.plane_depth;
        copy_box(ring + slot * kStage + kWeightBytes, &p.x, (x - plane * p.plane_depth) * kDepth, 0, plane,
                 &sh.full[slot]);
    };
    const int filled = min(last, first + (int)kRing);        // the ring's first turn
    if (warp == 0) {
        if (elect_one()) {
            for (uint32_t s = 0; s < kRing; ++s) bar_init(&sh.full[s], 1), bar_init(&sh.empty[s], 1);
            bar_init(&sh.done, 1);
            asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
            sh.fault = 0;
            sh.armed = 0;
            prefetch_map(&p.w);
            prefetch_map(&p.x);
            if (kSecond<FORM>)
                for (int x = first; x < filled; ++x) weights(x, (uint32_t)(x - first));
        }
        __syncwarp();
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&sh.tmem)),
                     "n"(kTmem)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
        fence_before();
    }
    pdl_enter();
    if (warp == 0) {
        if (elect_one()) {
            // the first product's results were stored by the launch before
            asm volatile("fence.proxy.async;" ::: "memory");
            for (int x = first; x < filled; ++x) {
                if (!kSecond<FORM>) weights(x, (uint32_t)(x - first));
                tokens(x, (uint32_t)(x - first));
            }
        }
        __syncwarp();
    }
    __syncthreads();
    fence_after();
    const uint32_t tmem = sh.tmem;

    if (warp == 0) {
        uint32_t slot = 0, turn = 0;
        int x = filled;
        for (; x < last; ++x) {
            if (!__all_sync(0xffffffffu, wait(sh, &sh.empty[slot], turn, p.wait_ns))) break;
            if (elect_one()) {
                weights(x, slot);
                tokens(x, slot);
            }
            __syncwarp();
            if (++slot == kRing) slot = 0, turn ^= 1;
        }
        if (lane == 0) sh.armed = (uint32_t)(x - first);
    }
    if (warp == 1) {
        uint32_t slot = 0, turn = 0;
        bool ok = true, ready = false;      // ready: the next stage is known to have landed
        const uint64_t desc_a = operand_at<kByRows>(ring, 0), desc_b = operand(ring + kWeightBytes);
        for (int x = first; x < last; ++x) {
            if (!ready) {
                ok = __all_sync(0xffffffffu, wait(sh, &sh.full[slot], turn, p.wait_ns));
                if (!ok) break;
            }
            fence_after();
            const uint64_t a = desc_a + slot * (kStage >> 4), t = desc_b + slot * (kStage >> 4);
            if (elect_one()) {
#pragma unroll
                for (int k = 0; k < kDepth / 16; ++k)
                    mma(tmem, a + k * ((kByRows ? 2048 : 32) >> 4), t + k * (32 >> 4), kKind, x > first || k > 0);
                commit(&sh.empty[slot]);
            }
            __syncwarp();
            if (++slot == kRing) slot = 0, turn ^= 1;
            ready = x + 1 < last && __all_sync(0xffffffffu, landed(smem_u32(&sh.full[slot]), turn));
        }
        if (elect_one()) commit(&sh.done);  // (after a wait that gave up, of what was started)
        __syncwarp();
        // by then every copy has been consumed, unless a wait gave up
        if (ok) wait(sh, &sh.done, 0, p.wait_ns);
    }
    __syncwarp();
    __syncthreads();
    if (sh.fault) {
        // A wait gave up: let what is in flight land before its memory is used
        // or given back; of a slot, the last stage tells.
        if (threadIdx.x < kRing && threadIdx.x < sh.armed) {
            const uint32_t turns = (sh.armed - 1 - threadIdx.x) / kRing;
            stage_wait(smem_u32(&sh.full[threadIdx.x]), turns & 1, globaltimer_ns() + kStageWaitNs, kStageWaitNs);
        }
        if (threadIdx.x == 32)
            stage_wait(smem_u32(&sh.done), 0, globaltimer_ns() + kStageWaitNs, kStageWaitNs);
        __syncwarp();
        __syncthreads();
    }
    // partial sums: [token][128] in place of the ring
    float* partial = (float*)(raw + (ring - smem_u32(raw)));
    if (warp >= 4 && !sh.fault) {
        fence_after();
        const uint32_t d = tmem + ((uint32_t)(warp & 3) << 21);
        float* mine = partial + (warp & 3) * 32 + lane;
#pragma unroll 1
        for (int n0 = 0; n0 < p.tokens; n0 += NT < 16 ? NT : 16) {
            float v[16], low[16];
            load_columns(d + n0, d + (!kSecond<FORM> || NT < 16 || kParts<NT> == 1 ? n0 : NT + n0), v, low);
#pragma unroll
            for (int n = 0; n < (NT < 16 ? NT : 16); ++n) {
                float sum = v[n];
                if constexpr (kSecond<FORM> && kParts<NT> == 2) {
                    // (a sum of lower parts that is not finite comes from a weight that is not: the upper parts' tells)
                    const float rest = NT < 16 ? v[n + NT < 16 ? n + NT : 0] : low[n];
                    if (isfinite(rest)) sum = fmaf(kLowUnit<T>, rest, sum);
                }
                if (n0 + n < p.tokens) mine[(n0 + n) * kRows] = sum;
            }
        }
        fence_before();
    }
    __syncwarp();
    cluster_sync();
    const int faults = threadIdx.x < p.split ? (int)remote_read(in_block(smem_u32(&sh.fault), threadIdx.x)) : 0;
    if (!__syncthreads_or(faults)) {
        constexpr int kItems = FORM == kIn ? kRows / 2 : kRows;
        const int items = (p.tokens + kAtOnce - 1) / kAtOnce * kItems, end = items * (rank + 1) / p.split;
        for (int i = items * rank / p.split + (int)threadIdx.x; i < end; i += kThreads) {
            const int t0 = i / kItems * kAtOnce, r = i % kItems, col = tile * kItems + r;
            if (col >= p.rows) continue;
            const int count = min(kAtOnce, p.tokens - t0);
            const uint32_t at = smem_u32(partial + t0 * kRows + r);
            float g[kAtOnce], u[kAtOnce], sum[kAtOnce];
            if constexpr (FORM == kBackIn)
#pragma unroll
                for (int j = 0; j < kAtOnce; ++j)
                    if (j < count) {
                        const T* pre = (const T*)p.pre + (t0 + j) * p.ld_pre + col;
                        g[j] = to_f32(pre[0]);
                        u[j] = to_f32(pre[p.inter]);
                    }
            sums_of_blocks(at, kRows * 4, count, p.split, sum);
            if constexpr (FORM == kIn) sums_of_blocks(at + kItems * 4, kRows * 4, count, p.split, u);
#pragma unroll
            for (int j = 0; j < kAtOnce; ++j) {
                if (j >= count) break;
                const int64_t t = t0 + j;
                T* to = (T*)p.out + t * p.ld_out + col;
                if constexpr (FORM == kIn) {
                    const Parts<T> h = split_parts<T>(act_value<ACT>(sum[j]) * u[j]);
                    to[0] = h.high;
                    if constexpr (kParts<NT> == 2) to[NT * p.ld_out] = h.low;
                    if (p.pre) {
                        T* pre = (T*)p.pre + t * p.ld_pre + col;
                        pre[0] = from_f32<T>(sum[j]);
                        pre[p.inter] = from_f32<T>(u[j]);
                    }
                } else if constexpr (FORM == kBackIn) {
                    const Act a = act_both<ACT>(g[j]);
                    const Parts<T> dg = split_parts<T>(sum[j] * u[j] * a.slope), du = split_parts<T>(sum[j] * a.value);
                    to[0] = dg.high;
                    to[p.plane] = du.high;
                    if constexpr (kParts<NT> == 2) {
                        to[NT * p.ld_out] = dg.low;
                        to[p.plane + NT * p.ld_out] = du.low;
                    }
                    ((T*)p.h)[t * p.ld_out + col] = from_f32<T>(a.value * u[j]);
                } else {
                    to[0] = from_f32<T>(sum[j]);
                }
            }
        }
    }
    __syncwarp();
    cluster_sync();                         // the others have read this block's sums
    if (warp == 1) {
        fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(kTmem) : "memory");
    }
}

// ---- host side ------------------------------------------------------------------------

template <class T, int FORM, int ACT, int NT>
cudaError_t launch(Params& p, int64_t rows, int64_t depth, cudaStream_t s)
{
    const int64_t per = FORM == kIn ? kRows / 2 : kRows, tiles = (rows + per - 1) / per;
    p.rows = (int32_t)rows;
    p.plane_depth = (int32_t)((depth + kDepth - 1) / kDepth);
    p.depth = FORM == kBackX ? 2 * p.plane_depth : p.plane_depth;
    // as many blocks as run at a time, each with a stage at least; more where a
    // block's sums would be longer than a chain (of the widest blocks two chains)
    int64_t split = kSlots / tiles;
    if (split < (p.depth + kChain - 1) / kChain) split = (p.depth + kChain - 1) / kChain;
    if (split > kMaxSplit) split = kMaxSplit;
    if (split > p.depth) split = p.depth;
    p.split = split < 1 ? 1 : (int32_t)split;
    p.wait_ns = copy_wait_ns();
    auto kernel = ffn_few_kernel<T, FORM, ACT, NT>;
    static std::atomic<uint64_t> done{0};
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(tiles * p.split));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSharedBytes<FORM, NT>;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)p.split, attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = programmatic_launch() ? 2 : 1;
    return launch_shared((const void*)kernel, (int)kSharedBytes<FORM, NT>, done,
                         [&] { return cudaLaunchKernelEx(&cfg, kernel, p); });
}

// A token matrix: a single row may have any pitch.
inline bool encode_tokens(CUtensorMap* map, const void* base, int64_t tokens, int64_t cols, int64_t ld, int box_rows,
                          bool f16)
{
    return encode_matrices(map, base, 1, tokens, cols, tokens > 1 ? ld : cols, box_rows, f16);
}

template <class T, int ACT, int NT>
cudaError_t forward(const FfnParams& q, cudaStream_t s)
{
    constexpr bool f16 = std::is_same<T, __half>::value;
    const int64_t ip = padded_inter(q.inter);
    Params p;
    memset(&p, 0, sizeof(p));
    p.tokens = (int32_t)q.tokens;
    p.inter = q.inter;
    p.out = q.ws, p.ld_out = ip;
    p.pre = q.pre, p.ld_pre = q.ld_pre;
    if (!encode_matrices(&p.w, q.w_in, 2, q.inter, q.hidden, q.ld_in, kRows / 2, f16) ||
        !encode_tokens(&p.x, q.x, q.tokens, q.hidden, q.ld_x, kColumns<kIn, NT>, f16))
        return cudaErrorNotSupported;
    const cudaError_t e = launch<T, kIn, ACT, NT>(p, q.inter, q.hidden, s);
    if (e != cudaSuccess) return e;
    p.out = q.y, p.ld_out = q.ld_y;
    if (!encode_matrices(&p.w, q.w_out, 1, q.hidden, q.inter, q.ld_out, kRows, f16) ||
        !encode_matrices(&p.x, q.ws, 1, kParts<NT> * NT, q.inter, ip, kColumns<kOut, NT>, f16))
        return cudaErrorNotSupported;
    return launch<T, kOut, 0, NT>(p, q.hidden, q.inter, s);
}

// dg, du and h into the workspace (BackLayout), and dx where it is asked for.
template <class T, int ACT, int NT>
cudaError_t backward(const FfnBackParams& q, cudaStream_t s)
{
    constexpr bool f16 = std::is_same<T, __half>::value;
    const BackLayout l = back_layout(q.tokens, q.inter);
    Params p;
    memset(&p, 0, sizeof(p));
    p.tokens = (int32_t)q.tokens;
    p.inter = q.inter;
    p.out = q.ws, p.ld_out = l.ld, p.plane = l.plane;
    p.h = (T*)q.ws + l.h;
    p.pre = (void*)q.pre, p.ld_pre = q.ld_pre;
    if (!encode_matrices(&p.w, q.w_out, 1, q.hidden, q.inter, q.ld_out, kDepth, f16) ||
        !encode_tokens(&p.x, q.dy, q.tokens, q.hidden, q.ld_dy, kColumns<kBackIn, NT>, f16))
        return cudaErrorNotSupported;
    const cudaError_t e = launch<T, kBackIn, ACT, NT>(p, q.inter, q.hidden, s);
    if (e != cudaSuccess || !q.dx) return e;
    p.out = q.dx, p.ld_out = q.ld_dx;
    if (!encode_matrices(&p.w, q.w_in, 2, q.inter, q.hidden, q.ld_in, kDepth, f16) ||
        !encode_planes(&p.x, q.ws, 2, kParts<NT> * NT, q.inter, l.ld, l.plane, 64, kColumns<kBackX, NT>, f16))
        return cudaErrorNotSupported;
    return launch<T, kBackX, 0, NT>(p, q.hidden, q.inter, s);
}

template <class T, int ACT>
cudaError_t forward(const FfnParams& q, cudaStream_t s)
{
    if (q.tokens <= 8) return forward<T, ACT, 8>(q, s);
    if (q.tokens <= 16) return forward<T, ACT, 16>(q, s);
    if (q.tokens <= 32) return forward<T, ACT, 32>(q, s);
    if (q.tokens <= 64) return forward<T, ACT, 64>(q, s);
    return forward<T, ACT, 128>(q, s);
}

template <class T, int ACT>
cudaError_t backward(const FfnBackParams& q, cudaStream_t s)
{
    if (q.tokens <= 8) return backward<T, ACT, 8>(q, s);
    if (q.tokens <= 16) return backward<T, ACT, 16>(q, s);
    if (q.tokens <= 32) return backward<T, ACT, 32>(q, s);
    if (q.tokens <= 64) return backward<T, ACT, 64>(q, s);
    return backward<T, ACT, 128>(q, s);
}

}  // namespace few

}  // namespace

}  // namespace ptoc
