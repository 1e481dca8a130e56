// A mixture-of-experts layer for up to 64 tokens in one cooperative launch on
// the tensor cores.
//
// Bound by HBM: the active experts' 3 * inter * hidden weights, read once.
// The kernel is therefore one stream of weight tiles through shared memory
// (tensor-map copies, a ring of stages deep enough to cover the latency of
// HBM) into tcgen05.mma, whose rows are rows of weights and whose columns are
// all the call's tokens, padded to N = 8, 16, 32, 48 or 64: an expert multiplies
// every token, and the epilogue keeps those that chose it. The second product
// has 2 N columns: the activations are split into an upper and a lower part of
// the type (moe_common.cuh), which the epilogue adds up. The tensor cores are
// nearly idle at any N (4 % busy at 1 token), so gathering tokens would save
// nothing that is short. A stage is 256 rows of weights (two accumulators of
// 128 rows) by 64 elements of depth, and the tokens' elements of that depth.
//
//   phase 0  logits in binary32 on the CUDA cores           | grid barrier
//   routing  few tokens: every block chooses for every token (the same bits
//            everywhere); more: one block per token         | grid barrier
//   phase 1  tiles of 128 gate rows and the matching 128 up rows x hidden;
//            epilogue: h[expert][token] = w * silu(gate) * up in its two
//            parts, zero for tokens that did not choose the
//            expert                                         | grid barrier
//            the same for tiles of several parts            | grid barrier
//   phase 2  tiles of 256 output columns x (inter of every active expert):
//            the sum over experts stays in the accumulator  | grid barrier
//            sums of tiles of several parts
//
// Work is split evenly in units of one stage: block c takes the stages
// [c, c + 1) * total / blocks, in tile order, so that a tile may be spread over
// several blocks. Those write binary32 partial tiles, which all blocks together
// add after a barrier, in the order of the parts: the sum does not depend on
// scheduling. (Added by the block that comes last at a tile, without the
// barrier, 3 parts of 64 tokens took 22 us instead of 3.) The weights of phase
// 2's first stages are on their way before the barriers in front of it.
//
// Measured on GB300 (bf16, of 6.79 TB/s copied): 64 tokens x 128 experts of 4096
// x 1536 751 to 780 us from GPU to GPU (6.3 to 6.1 TB/s); 32 tokens 642 us; 1
// token, 8 of 64 experts of 7168 x 2048, 128 us (5.5 TB/s); 1 token, 8 of 128 of
// 4096 x 1536, 71 us (4.2 TB/s); 64 tokens x 16 experts of 1024 x 512 38 us
// (floor 8: nearly every tile is in parts). With one rounded activation in
// place of two parts 64 tokens took 729 us where these took 751, 32 tokens 632
// and one token the same: half of that is the ring's stage that the second part
// takes, half its passing L2 with every tile of weights. What a call costs
// beside its stream of weights is 25 us at 1 token and 50 to 80 us at 64: four
// grid barriers (five with more than 8 tokens) of 1.2 us, the latency of the
// first copies of either phase (3 us each), the choice (2 us), the epilogues,
// and at 64 tokens the partial tiles and both parts.
// Stages of 128 rows (two per tile of gate and up rows) took 829 us at 64 tokens
// when these took 756, as the tokens' elements then pass L2 twice as often;
// boxes without promotion to 256 bytes in L2 872 us; stages of 128 elements of
// depth the same as 64.
#include <cooperative_groups.h>

#include "host/host_checks.h"
#include "layers/moe_common.cuh"
#include "reduce_forms.cuh"

namespace ptoc {

namespace {

namespace cg = cooperative_groups;

constexpr int kDepth = 64;                  // one stage: 64 elements (128 bytes, one swizzle row) of K
constexpr int kHalfRows = 128;              // rows of one accumulator
constexpr int kTileRows = 2 * kHalfRows;    // phase 1: gate and up rows; phase 2: output columns
constexpr int kHalfBytes = kHalfRows * kDepth * 2;
constexpr int kTileBytes = 2 * kHalfBytes;
constexpr int kThreads = 256;               // warp 0 copies, warp 1 multiplies, warps 4 to 7 drain
constexpr int kWarps = kThreads / 32;
constexpr int kEpilogue = 128;
constexpr int kMaxStages = 8;

struct MoeTensorParams {
    CUtensorMap w_in, w_out, x, h;
    MoeParams m;
    float* logits;                          // [tokens, experts]
    char* act;                              // [active, 2 N, inter] activations, their upper and lower parts (the h map)
    float* partial;                         // [2 * grid][2][tokens][128] binary32 partial tiles
    uint32_t* bad;                          // [tiles of phase 2] 1: of several parts, over weights that are not finite
    int32_t* ids;                           // [tokens, top_k], where one block chooses per token
    float* weights;
    uint64_t wait_ns;
};

constexpr int kGrid = 152;                  // one block per SM; the workspace is sized for it

// A tile of several parts, which the blocks c0 to c1 hold.
struct PartedTile {
    uint32_t tile;
    uint16_t c0, c1;
};

// ---- shared memory ----------------------------------------------------------------

struct Shared {
    uint64_t full[kMaxStages], empty[kMaxStages];
    uint64_t acc_full[2], acc_empty[2], drained;
    uint32_t tmem;
    int32_t active;                         // active local experts
    int32_t fault;                          // a bounded wait gave up
    uint32_t armed;                         // stages whose copies were started, over both phases
    int32_t ids[PTOC_MOE_MAX_TOKENS * PTOC_MOE_MAX_TOP_K];
    float weights[PTOC_MOE_MAX_TOKENS * PTOC_MOE_MAX_TOP_K];
    int16_t expert[PTOC_MOE_MAX_EXPERTS];   // the active local experts, ascending
    PartedTile parted[2][kGrid];            // the tiles of several parts of either phase
    int32_t parted_tiles[2];
    float row_weight[PTOC_MOE_MAX_TOKENS];  // of the epilogue's expert
    int32_t chosen[PTOC_MOE_MAX_TOKENS];
    union {
        float dots[kWarps][16];
        uint32_t bits[PTOC_MOE_MAX_EXPERTS / 32];
    };
};

constexpr size_t kSharedHead = (sizeof(Shared) + 1023) / 1024 * 1024;
// The call's tokens are padded to N = 8, 16, 32, 48 or 64. The first product
// multiplies them as they are (with the 16 columns that an mma has at least),
// the second one both parts of their activations.
template <int N>
constexpr int kInColumns = N < 16 ? 16 : N;
template <int N>
constexpr int kOutColumns = 2 * N;
constexpr int kRowBytes = kDepth * 2;
template <int N>
constexpr uint32_t kStageBytes = kTileBytes + kOutColumns<N> * kRowBytes;
constexpr size_t kSharedMost = 227 * 1024;
// stages of the ring: what the head, and room to align it, leave
template <int N>
constexpr int kRing = (int)((kSharedMost - kSharedHead - 1024) / kStageBytes<N>) < kMaxStages
                          ? (int)((kSharedMost - kSharedHead - 1024) / kStageBytes<N>)
                          : kMaxStages;

// ---- tensor-core and copy instructions ------------------------------------------------

// A K-major operand of 128-byte rows in the 128-byte swizzle: groups of 8 rows
// are 1024 bytes apart.
__device__ __forceinline__ uint64_t operand(uint32_t addr)
{
    return (uint64_t)((addr & 0x3ffffu) >> 4) | (uint64_t)1 << 16 | (uint64_t)(1024 >> 4) << 32 | (uint64_t)1 << 46 |
           (uint64_t)2 << 61;
}

__device__ __forceinline__ void mma(uint32_t d, uint64_t a, uint64_t b, uint32_t kind, uint32_t accumulate)
{
    asm volatile("{ .reg .pred p; setp.ne.u32 p, %4, 0;\n"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p; }"
                 ::"r"(d), "l"(a), "l"(b), "r"(kind), "r"(accumulate)
                 : "memory");
}

// The barrier completes when every mma issued so far by this thread has.
__device__ __forceinline__ void commit(uint64_t* bar)
{
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar))
                 : "memory");
}

// Sixteen columns of both halves of an accumulator, this thread's row.
__device__ __forceinline__ void load_columns(uint32_t lo_at, uint32_t hi_at, float (&lo)[16], float (&hi)[16])
{
    // (one statement: nothing may use the columns before the wait)
    uint32_t u[16], v[16];
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 "
                 "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%32];\n"
                 "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
                 "{%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%33];\n"
                 "tcgen05.wait::ld.sync.aligned;"
                 : "=&r"(u[0]), "=&r"(u[1]), "=&r"(u[2]), "=&r"(u[3]), "=&r"(u[4]), "=&r"(u[5]), "=&r"(u[6]),
                   "=&r"(u[7]), "=&r"(u[8]), "=&r"(u[9]), "=&r"(u[10]), "=&r"(u[11]), "=&r"(u[12]), "=&r"(u[13]),
                   "=&r"(u[14]), "=&r"(u[15]), "=&r"(v[0]), "=&r"(v[1]), "=&r"(v[2]), "=&r"(v[3]), "=&r"(v[4]),
                   "=&r"(v[5]), "=&r"(v[6]), "=&r"(v[7]), "=&r"(v[8]), "=&r"(v[9]), "=&r"(v[10]), "=&r"(v[11]),
                   "=&r"(v[12]), "=&r"(v[13]), "=&r"(v[14]), "=&r"(v[15])
                 : "r"(lo_at), "r"(hi_at)
                 : "memory");
#pragma unroll
    for (int i = 0; i < 16; ++i) lo[i] = __uint_as_float(u[i]), hi[i] = __uint_as_float(v[i]);
}

// f(0) to f(min(count, N) - 1), without a branch between them where all are asked for.
template <int N, class F>
__device__ __forceinline__ void each(int count, F f)
{
    if (count >= N) {
#pragma unroll
        for (int n = 0; n < N; ++n) f(n);
    } else {
#pragma unroll
        for (int n = 0; n < N; ++n)
            if (n < count) f(n);
    }
}

__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

__device__ __forceinline__ void bar_init(uint64_t* bar, uint32_t count)
{
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(bar)), "r"(count) : "memory");
}

__device__ __forceinline__ void bar_arrive(uint64_t* bar)
{
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}

__device__ __forceinline__ void bar_expect(uint64_t* bar, uint32_t bytes)
{
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(smem_u32(bar)), "r"(bytes) : "memory");
}

// A box of a tensor map at column x (a multiple of 64 elements) and row y of matrix z.
__device__ __forceinline__ void copy_box(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint64_t* bar)
{
    asm volatile("cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
                 "[%0], [%1, {%2, %3, %4}], [%5];"
                 ::"r"(dst), "l"(map), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
                 : "memory");
}

__device__ __forceinline__ void epilogue_sync() { asm volatile("bar.sync 1, %0;" ::"n"(kEpilogue) : "memory"); }

// ---- the split of the work ----------------------------------------------------------

// `total` stages, `depth` of them to a tile, over `blocks` blocks.
struct Split {
    uint32_t total, depth;
    uint32_t blocks;                        // at most `total`: every one has work
    __device__ Split(uint32_t tiles, uint32_t d, uint32_t grid)
        : total(tiles * d), depth(d), blocks(tiles * d < grid ? tiles * d : grid) {}
    __device__ uint32_t begin(uint32_t c) const
    {
        return c >= blocks ? total : (uint32_t)((uint64_t)c * total / blocks);
    }
    // the block that holds stage x: the largest c with begin(c) <= x
    __device__ uint32_t owner(uint32_t x) const { return (uint32_t)((((uint64_t)x + 1) * blocks - 1) / total); }
    // Tiles of several parts are those that a block other than the first begins
    // within. Whether block c >= 1 is the first to begin within its tile.
    __device__ bool parted(uint32_t c, PartedTile& t) const
    {
        const uint32_t x = begin(c);
        t.tile = x / depth;
        if (x == t.tile * depth || begin(c - 1) > t.tile * depth) return false;
        t.c0 = (uint16_t)(c - 1);
        t.c1 = (uint16_t)owner((t.tile + 1) * depth - 1);
        return true;
    }
};

// A bounded wait on a barrier of this block; false once any wait of the block
// gave up, and then for good: the places in the ring go on by what a phase
// should have done, so the parity of a later wait could be that of a turn which
// its barrier never saw, and a stage would be armed twice. (The same by a flag
// in a register of each role cost 4 us a call.) The clock is read only after a
// number of polls (each of which may be suspended for a while): read by all SMs
// at once it takes a microsecond or more.
__device__ __forceinline__ bool wait(Shared& sh, uint64_t* bar, uint32_t parity, uint64_t bound_ns)
{
    constexpr int kPolls = 64;
    if (*(volatile int32_t*)&sh.fault) return false;
    for (int i = 0; i < kPolls; ++i)
        if (stage_ready(smem_u32(bar), parity)) return true;
    if (stage_wait(smem_u32(bar), parity, globaltimer_ns() + bound_ns, bound_ns)) return true;
    if (atomicExch(&sh.fault, 1) == 0) atomicAdd(&g_stage_faults, 1u);
    return false;
}

// The same wait by the epilogue's threads, which go on or stop together.
__device__ __forceinline__ bool epilogue_wait(Shared& sh, uint64_t* bar, uint32_t parity, uint64_t bound_ns)
{
    uint32_t all;
    asm volatile("{ .reg .pred p, q; setp.ne.u32 p, %1, 0; bar.red.and.pred q, 1, %2, p; selp.u32 %0, 1, 0, q; }"
                 : "=r"(all)
                 : "r"((uint32_t)wait(sh, bar, parity, bound_ns)), "n"(kEpilogue)
                 : "memory");
    return all != 0;
}

// ---- phase 0 ----------------------------------------------------------------------

template <class T>
__device__ __forceinline__ F8 load_router8(const void* base, bool f32, int64_t i)
{
    if (f32) {
        const float4 a = *(const float4*)((const float*)base + i), b = *(const float4*)((const float*)base + i + 4);
        return F8{pair(a.x, a.y), pair(a.z, a.w), pair(b.x, b.y), pair(b.z, b.w)};
    }
    return load8<T, 8>((const T*)base + i, 0, 1).expand();
}

// Dot products of ET experts with TT tokens per block and turn (ET * TT is a
// power of two of at most 16); the warps share the rows and their sums are
// added in order.
template <class T, int ET, int TT>
__device__ __forceinline__ void router_logits(const MoeTensorParams& p, Shared& sh)
{
    constexpr int kSums = ET * TT;
    const MoeParams& m = p.m;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int groups = (m.tokens + TT - 1) / TT;
    const int units = (m.experts + ET - 1) / ET * groups;
    // Every block takes a turn, though there may be fewer units than blocks (the
    // answers of the extra turns are dropped): a block that has slept until the
    // barrier takes 3 us longer over the choice that follows.
    for (int turn = blockIdx.x; turn < max(units, (int)gridDim.x); turn += gridDim.x) {
        const int u = turn % units;
        const int e0 = u / groups * ET, t0 = u % groups * TT;
        Pair sum[ET][TT] = {};
        // tokens and experts past the last are computed as the last and dropped
#pragma unroll(kSums > 4 ? 2 : 4)
        for (int64_t i = threadIdx.x * 8; i < m.hidden; i += kThreads * 8) {
            F8 r[ET];
#pragma unroll
            for (int e = 0; e < ET; ++e)
                r[e] = load_router8<T>(m.router, m.router_f32, (int64_t)min(e0 + e, m.experts - 1) * m.hidden + i);
#pragma unroll
            for (int t = 0; t < TT; ++t) {
                const F8 x = load_router8<T>(m.x, false, min(t0 + t, m.tokens - 1) * m.ld_x + i);
#pragma unroll
                for (int e = 0; e < ET; ++e)
#pragma unroll
                    for (int j = 0; j < 4; ++j) sum[e][t] = fma2(r[e].p[j], x.p[j], sum[e][t]);
            }
        }
        // kSums sums over 32 lanes: each exchange halves the values that a lane
        // keeps, until it keeps one; then the lanes that keep the same add up
        float v[kSums];
#pragma unroll
        for (int i = 0; i < kSums; ++i) v[i] = sum_of(sum[i / TT][i % TT]);
        int o = 16;
#pragma unroll
        for (int n = kSums / 2; n >= 1; n >>= 1, o >>= 1) {
            const bool upper = lane & o;
#pragma unroll
            for (int i = 0; i < n; ++i) {
                const float give = upper ? v[i] : v[n + i], keep = upper ? v[n + i] : v[i];
                v[i] = keep + __shfl_xor_sync(0xffffffffu, give, o);
            }
        }
        constexpr int kSame = 32 / kSums;                    // neighbouring lanes that keep the same sum
        for (; o >= 1; o >>= 1) v[0] += __shfl_xor_sync(0xffffffffu, v[0], o);
        if (lane % kSame == 0) sh.dots[warp][lane / kSame] = v[0];
        __syncthreads();
        if (threadIdx.x < kSums) {
            float d = 0.0f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) d += sh.dots[w][threadIdx.x];
            const int e = e0 + threadIdx.x / TT, t = t0 + threadIdx.x % TT;
            if (turn < units && e < m.experts && t < m.tokens) p.logits[t * m.experts + e] = d;
        }
        __syncthreads();
    }
}

__device__ __forceinline__ void choose(const MoeParams& m, const float* logits, int32_t* ids, float* weights)
{
    if (m.experts <= 128) choose_experts<4>(m, logits, ids, weights);
    else choose_experts<32>(m, logits, ids, weights);
}

// The choice of every token, and the list of active local experts. One choice
// takes a warp about 1 us: up to kThreads / 32 tokens are chosen for in every
// block, more by one block each and one more grid barrier (about 2 us).
__device__ __forceinline__ void route(const MoeTensorParams& p, Shared& sh, const cg::grid_group& grid)
{
    const MoeParams& m = p.m;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int pairs = m.tokens * m.top_k;
    if (m.tokens <= kThreads / 32) {
        if (warp < m.tokens)
            choose(m, p.logits + warp * m.experts, sh.ids + warp * m.top_k, sh.weights + warp * m.top_k);
    } else {
        if (warp == 0)
            for (int t = blockIdx.x; t < m.tokens; t += gridDim.x)
                choose(m, p.logits + t * m.experts, p.ids + t * m.top_k, p.weights + t * m.top_k);
        grid.sync();
        for (int i = threadIdx.x; i < pairs; i += kThreads) {
            sh.ids[i] = p.ids[i];
            sh.weights[i] = p.weights[i];
        }
    }
    if (threadIdx.x < PTOC_MOE_MAX_EXPERTS / 32) sh.bits[threadIdx.x] = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < pairs; i += kThreads) {
        const int local = sh.ids[i] - m.first;
        if (local >= 0 && local < m.local) atomicOr(&sh.bits[local >> 5], 1u << (local & 31));
        if (blockIdx.x == 0) {
            if (m.ids) m.ids[i] = sh.ids[i];
            if (m.weights) m.weights[i] = sh.weights[i];
        }
    }
    __syncthreads();
    if (warp == 0) {
        uint32_t mine = sh.bits[lane];
        int before = __popc(mine), all = before;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, all, o);
            if (lane >= o) all += v;
        }
        before = all - before;
        for (; mine; mine &= mine - 1) sh.expert[before++] = (int16_t)(lane * 32 + __ffs(mine) - 1);
        if (lane == 31) sh.active = all;
    }
    __syncthreads();
}

// ---- tiles ------------------------------------------------------------------------

// One element of h.
__device__ __forceinline__ float activation(float w, float gate, float up)
{
    return w * (gate / (1.0f + expf(-gate))) * up;
}

// The weight with which token t chose `expert`; false if it did not.
__device__ __forceinline__ bool chosen(const MoeParams& m, const Shared& sh, int t, int expert, float& w)
{
    bool hit = false;
    for (int k = 0; k < m.top_k; ++k)
        if (sh.ids[t * m.top_k + k] == expert) hit = true, w = sh.weights[t * m.top_k + k];
    return hit;
}

// The sums, in order, of the parts c0..c1 of a tile, for one token and the
// rows quad..quad+3 of both halves.
__device__ __forceinline__ void add_parts(const MoeTensorParams& p, uint32_t c0, uint32_t c1, int t, int quad,
                                          float4& lo, float4& hi)
{
    constexpr int kAtOnce = 8;
    const int64_t half = (int64_t)p.m.tokens * kHalfRows;
    lo = hi = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    auto add = [](float4& s, const float4& v) { s.x += v.x, s.y += v.y, s.z += v.z, s.w += v.w; };
    for (uint32_t c = c0; c <= c1; c += kAtOnce) {
        float4 v[kAtOnce][2];
#pragma unroll
        for (int q = 0; q < kAtOnce; ++q)
            if (c + q <= c1) {
                const int64_t slot = 2 * (int64_t)(c + q) + (c + q == c0);
                const float* part = p.partial + slot * 2 * half + t * kHalfRows + quad;
                v[q][0] = __ldcg((const float4*)part);
                v[q][1] = __ldcg((const float4*)(part + half));
            }
#pragma unroll
        for (int q = 0; q < kAtOnce; ++q)
            if (c + q <= c1) {
                add(lo, v[q][0]);
                add(hi, v[q][1]);
            }
    }
}

// Four neighbouring elements of a row of `n`, from column `col` on.
template <class T>
__device__ __forceinline__ void store4(T* row, int64_t col, int64_t n, const float4& v)
{
    const float e[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < 4; ++j)
        if (col + j < n) row[col + j] = from_f32<T>(e[j]);
}

// y of one token and column from the token's own experts alone, by a warp: the
// lanes share each expert's elements, and their sums are added in order.
template <class T, int N>
__device__ __noinline__ float own_sum(const MoeTensorParams& p, const Shared& sh, int t, int64_t col)
{
    const MoeParams& m = p.m;
    const int lane = threadIdx.x & 31;
    float sum = 0.0f;
    for (int a0 = 0; a0 < sh.active; a0 += 32) {
        float w;
        const bool hit = a0 + lane < sh.active && chosen(m, sh, t, m.first + sh.expert[a0 + lane], w);
        for (uint32_t hits = __ballot_sync(0xffffffffu, hit); hits; hits &= hits - 1) {
            const int a = a0 + __ffs(hits) - 1;
            const unsigned short* h = (const unsigned short*)p.act + ((int64_t)a * 2 * N + t) * m.inter;
            const unsigned short* low = h + N * m.inter;
            const T* row = (const T*)m.w_out + ((int64_t)sh.expert[a] * m.hidden + col) * m.inter;
#pragma unroll 4
            for (int64_t i = lane; i < m.inter; i += 32) {
                const Parts<T> v{bitcast<T>((uint16_t)__ldcg(h + i)), bitcast<T>((uint16_t)__ldcg(low + i))};
                sum = fmaf(v.value(), to_f32(row[i]), sum);
            }
        }
    }
    return warp_sum(sum);
}

// The sums of phase 2 run over the experts of all tokens, with an activation
// of 0 for those that a token did not choose: an infinity or a NaN in the
// w_out of such an expert makes them NaN. Sums over such weights are taken
// again, for tokens [t0, t1) of this lane's column if its weights are `bad`; the
// warp does it together, for one lane after the other. What tells is the sum of
// any token's lower parts: they are finite whatever the activations are, so it
// is finite unless a weight is not. (Asked of y instead, calls with finite
// weights and one f16 activation beyond the range took 108 ms instead of 0.24:
// 64 tokens, 4 of 8 experts of 40960 x 512. A tile may not take longer than the
// other roles wait for it.)
template <class T, int N>
__device__ __forceinline__ void mend(const MoeTensorParams& p, const Shared& sh, bool bad, int t0, int t1, int64_t col)
{
    const int lane = threadIdx.x & 31;
    for (uint32_t all = __ballot_sync(0xffffffffu, bad && col < p.m.hidden); all; all &= all - 1) {
        const int src = __ffs(all) - 1;
        const int64_t c = __shfl_sync(0xffffffffu, col, src);
        for (int t = t0; t < t1; ++t) {
            const float sum = own_sum<T, N>(p, sh, t, c);
            if (lane == src) ((T*)p.m.y)[t * p.m.ld_y + c] = from_f32<T>(sum);
        }
    }
}

template <class T, int N>
__global__ void __launch_bounds__(kThreads, 1) moe_tensor_kernel(const __grid_constant__ MoeTensorParams p)
{
    extern __shared__ unsigned char raw[];
    Shared& sh = *(Shared*)raw;
    const uint32_t ring = (smem_u32(raw) + (uint32_t)kSharedHead + 1023u) & ~1023u;
    constexpr uint32_t kStage = kStageBytes<N>;
    constexpr uint32_t kStages = kRing<N>;
    constexpr int kIn = kInColumns<N>, kOut = kOutColumns<N>;
    constexpr uint32_t kColumns = 4 * kOut;                  // two accumulators in turn, of two halves
    constexpr uint32_t kTmem = kColumns <= 64 ? 64 : kColumns <= 128 ? 128 : kColumns <= 256 ? 256 : 512;
    // f32 accumulator, both operands T, both K-major, 128 rows
    constexpr uint32_t kType = std::is_same<T, __half>::value ? 0u : 1u;
    constexpr uint32_t kKind = 1u << 4 | kType << 7 | kType << 10 | (kHalfRows >> 4) << 24;
    const MoeParams& m = p.m;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const cg::grid_group grid = cg::this_grid();

    if (threadIdx.x == 0) {
        for (uint32_t s = 0; s < kStages; ++s) bar_init(&sh.full[s], 1), bar_init(&sh.empty[s], 1);
        for (int b = 0; b < 2; ++b) bar_init(&sh.acc_full[b], 1), bar_init(&sh.acc_empty[b], kEpilogue);
        bar_init(&sh.drained, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        sh.fault = 0;
        sh.armed = 0;
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&sh.tmem)),
                     "n"(kTmem)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
        fence_before();
    }
    for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i * kTileRows < m.hidden;
         i += (int64_t)gridDim.x * kThreads)
        p.bad[i] = 0;
    // one or two tokens: all loads of a row at once, an expert to a block
    if (m.tokens <= 2) router_logits<T, 1, 2>(p, sh);
    else router_logits<T, 2, 8>(p, sh);
    grid.sync();
    fence_after();
    route(p, sh, grid);

    const uint32_t active = (uint32_t)sh.active;
    const uint32_t in_depth = (uint32_t)((m.hidden + kDepth - 1) / kDepth);
    const uint32_t out_depth = (uint32_t)((m.inter + kDepth - 1) / kDepth);
    const uint32_t in_tiles = (uint32_t)((m.inter + kHalfRows - 1) / kHalfRows);
    const uint32_t out_tiles = (uint32_t)((m.hidden + kTileRows - 1) / kTileRows);
    const Split in(active * in_tiles, in_depth, gridDim.x), out(out_tiles, active * out_depth, gridDim.x);
    const uint32_t tmem = sh.tmem;
    if (active == 0) {                      // nothing is held here: rows of zeros
        for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < m.tokens * m.hidden;
             i += (int64_t)gridDim.x * kThreads)
            ((T*)m.y)[i / m.hidden * m.ld_y + i % m.hidden] = from_f32<T>(0.0f);
    }

    // warps 2 and 3 list the tiles of several parts while the others begin (each
    // in the same order: the places are those of the blocks)
    if (warp == 2 || warp == 3) {
        const Split& split = warp == 2 ? in : out;
        int n = 0;
        for (uint32_t c0 = 1; c0 < split.blocks; c0 += 32) {
            PartedTile t;
            const bool on = c0 + lane < split.blocks && split.parted(c0 + lane, t);
            const uint32_t all = __ballot_sync(0xffffffffu, on);
            if (on) sh.parted[warp - 2][n + __popc(all & ((1u << lane) - 1))] = t;
            n += __popc(all);
        }
        if (lane == 0) sh.parted_tiles[warp - 2] = n;
    }

    // the roles' places in the ring and in the two accumulators, kept over both phases
    uint32_t turn = 0, acc = 0;
    for (int phase = 1; phase <= 2 && active > 0; ++phase) {
        const Split& split = phase == 1 ? in : out;
        const uint32_t first = split.begin(blockIdx.x), last = split.begin(blockIdx.x + 1);
        const uint32_t columns = phase == 1 ? kIn : kOut;
        // Copies of stage x: the weights' tile, then the tokens' rows of the same depth.
        auto weights = [&](uint32_t x, uint32_t slot) {
            const uint32_t tile = x / split.depth, d = x - tile * split.depth;
            const uint32_t dst = ring + slot * kStage;
            uint64_t* bar = &sh.full[slot];
            bar_expect(bar, kTileBytes + columns * kRowBytes);
            ++sh.armed;
            if (phase == 1) {
                const uint32_t a = tile / in_tiles;
                const int i0 = (int)(tile - a * in_tiles) * kHalfRows, e = 2 * sh.expert[a];
                copy_box(dst, &p.w_in, (int)d * kDepth, i0, e, bar);
                copy_box(dst + kHalfBytes, &p.w_in, (int)d * kDepth, i0, e + 1, bar);
            } else {
                const uint32_t a = d / out_depth, k = d - a * out_depth;
                const int h0 = (int)tile * kTileRows, e = sh.expert[a];
                copy_box(dst, &p.w_out, (int)k * kDepth, h0, e, bar);
                copy_box(dst + kHalfBytes, &p.w_out, (int)k * kDepth, h0 + kHalfRows, e, bar);
            }
        };
        auto tokens = [&](uint32_t x, uint32_t slot) {
            const uint32_t d = x % split.depth;
            const uint32_t dst = ring + slot * kStage + kTileBytes;
            if (phase == 1) {
                copy_box(dst, &p.x, (int)d * kDepth, 0, 0, &sh.full[slot]);
            } else {
                const uint32_t a = d / out_depth, k = d - a * out_depth;
                copy_box(dst, &p.h, (int)k * kDepth, 0, (int)a, &sh.full[slot]);
            }
        };
        uint32_t sent = 0;
        if (phase == 2) {
            // the first weights do not wait for the other blocks
            if (warp == 0) {
                if (lane == 0)
                    for (const uint32_t ahead = min(kStages, last - first); sent < ahead; ++sent) {
                        const uint32_t u = turn + sent;
                        if (!wait(sh, &sh.empty[u % kStages], (u / kStages & 1) ^ 1, p.wait_ns)) break;
                        weights(first + sent, u % kStages);
                    }
                __syncwarp();
            }
            grid.sync();
            // h of the tiles of several parts: a warp takes 128 rows for one token
            const uint32_t pairs = (uint32_t)(sh.parted_tiles[0] * m.tokens);
            for (uint32_t u = blockIdx.x * kWarps + warp; u < pairs; u += gridDim.x * kWarps) {
                const uint32_t i = u / (uint32_t)m.tokens;
                const int t = (int)(u - i * (uint32_t)m.tokens), quad = lane * 4;
                const PartedTile part = sh.parted[0][i];
                const uint32_t a = part.tile / in_tiles;
                float4 lo, hi;
                float w = 0.0f;
                if (chosen(m, sh, t, m.first + sh.expert[a], w)) {
                    add_parts(p, part.c0, part.c1, t, quad, lo, hi);
                    lo = make_float4(activation(w, lo.x, hi.x), activation(w, lo.y, hi.y), activation(w, lo.z, hi.z),
                                     activation(w, lo.w, hi.w));
                } else {
                    lo = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                }
                const Parts<T> v[4] = {split_parts<T>(lo.x), split_parts<T>(lo.y), split_parts<T>(lo.z),
                                       split_parts<T>(lo.w)};
                T* row = (T*)p.act + ((int64_t)a * 2 * N + t) * m.inter;
                const int64_t col = (int64_t)(part.tile - a * in_tiles) * kHalfRows + quad;
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (col + j < m.inter) row[col + j] = v[j].high, row[N * m.inter + col + j] = v[j].low;
            }
            // h, here and in the epilogue, was written with ordinary stores, and is
            // read by the tensor-map copies after the barrier
            asm volatile("fence.proxy.async;" ::: "memory");
            grid.sync();
        }
        if (warp == 0 && lane == 0) {
            for (uint32_t s = 0; s < sent; ++s) tokens(first + s, (turn + s) % kStages);
            for (uint32_t x = first + sent; x < last; ++x) {
                const uint32_t u = turn + (x - first);
                if (!wait(sh, &sh.empty[u % kStages], (u / kStages & 1) ^ 1, p.wait_ns)) break;
                weights(x, u % kStages);
                tokens(x, u % kStages);
            }
        }

        if (warp == 1 && lane == 0) {
            uint32_t at = acc;
            bool ok = true;
            for (uint32_t x = first; x < last && ok;) {
                // one segment: this block's stages of one tile
                const uint32_t end = min(last, (x / split.depth + 1) * split.depth);
                const uint32_t b = at & 1, d = tmem + b * 2 * kOut;
                const uint32_t kind = kKind | columns >> 3 << 17;
                if (!wait(sh, &sh.acc_empty[b], (at >> 1 & 1) ^ 1, p.wait_ns)) break;
                fence_after();
                for (const uint32_t from = x; x < end; ++x) {
                    const uint32_t u = turn + (x - first), slot = u % kStages;
                    ok = wait(sh, &sh.full[slot], u / kStages & 1, p.wait_ns);
                    if (!ok) break;
                    fence_after();
                    const uint32_t a = ring + slot * kStage;
#pragma unroll
                    for (int k = 0; k < kDepth / 16; ++k) {
                        const uint64_t tok = operand(a + kTileBytes + k * 32);
                        mma(d, operand(a + k * 32), tok, kind, x > from || k > 0);
                        mma(d + kOut, operand(a + kHalfBytes + k * 32), tok, kind, x > from || k > 0);
                    }
                    commit(&sh.empty[slot]);
                }
                if (ok) commit(&sh.acc_full[b]);
                ++at;
            }
        }

        if (warp >= 4) {
            const int row = threadIdx.x - 128;                       // of either half
            uint32_t at = acc;
            for (uint32_t x = first; x < last;) {
                const uint32_t tile = x / split.depth, head = tile * split.depth;
                const uint32_t end = min(last, head + split.depth);
                const bool whole = x == head && end == head + split.depth;
                const uint32_t b = at & 1, a = tile / in_tiles;      // a: the expert, in phase 1
                const int64_t i0 = (int64_t)(tile - a * in_tiles) * kHalfRows, col0 = (int64_t)tile * kTileRows;
                T* h = (T*)p.act + (int64_t)a * 2 * N * m.inter;
                if (phase == 1) {
                    const int expert = m.first + sh.expert[a];
                    float w = 0.0f;
                    if (row < m.tokens) {
                        sh.chosen[row] = chosen(m, sh, row, expert, w);
                        sh.row_weight[row] = w;
                    }
                }
                if (!epilogue_wait(sh, &sh.acc_full[b], at >> 1 & 1, p.wait_ns)) break;
                fence_after();
                const uint32_t d = tmem + b * 2 * kOut + ((uint32_t)(warp & 3) << 21);
                float* mine = p.partial + (2 * (int64_t)blockIdx.x + (x == head)) * 2 * m.tokens * kHalfRows + row;
#pragma unroll 1
                for (int n0 = 0; n0 < m.tokens; n0 += 16) {
                    float lo[16], hi[16];
                    load_columns(d + n0, d + kOut + n0, lo, hi);
                    float low_lo = 0.0f, low_hi = 0.0f;              // those of the first token
                    if (phase == 2) {                                // the lower parts' sums
                        if constexpr (N == 8) {
                            low_lo = lo[8], low_hi = hi[8];
#pragma unroll
                            for (int n = 0; n < 8; ++n) {
                                lo[n] = fmaf(kLowUnit<T>, lo[n + 8], lo[n]);
                                hi[n] = fmaf(kLowUnit<T>, hi[n + 8], hi[n]);
                            }
                        } else {
                            float u[16], v[16];
                            load_columns(d + N + n0, d + kOut + N + n0, u, v);
                            low_lo = u[0], low_hi = v[0];
#pragma unroll
                            for (int n = 0; n < 16; ++n) {
                                lo[n] = fmaf(kLowUnit<T>, u[n], lo[n]);
                                hi[n] = fmaf(kLowUnit<T>, v[n], hi[n]);
                            }
                        }
                    }
                    const int count = m.tokens - n0;                 // columns that are tokens
                    if (!whole) {
                        float* to = mine + n0 * kHalfRows;
                        each<16>(count, [&](int n) { to[n * kHalfRows] = lo[n]; });
                        to += m.tokens * kHalfRows;
                        each<16>(count, [&](int n) { to[n * kHalfRows] = hi[n]; });
                        if (phase == 2 && !isfinite(low_lo + low_hi)) p.bad[tile] = 1;
                    } else if (phase == 1) {
                        // of an expert that the token did not choose it is 0, whatever the sums hold
                        T* to = h + (int64_t)n0 * m.inter + i0 + row;
                        if (i0 + row < m.inter)
                            each<16>(count, [&](int n) {
                                const int t = n0 + n;
                                const Parts<T> v =
                                    split_parts<T>(sh.chosen[t] ? activation(sh.row_weight[t], lo[n], hi[n]) : 0.0f);
                                to[n * m.inter] = v.high;
                                to[(n + N) * m.inter] = v.low;
                            });
                    } else {
                        auto put = [&](const float (&v)[16], float low, int64_t col) {
                            if (col < m.hidden) {
                                T* to = (T*)m.y + n0 * m.ld_y + col;
                                each<16>(count, [&](int n) { to[n * m.ld_y] = from_f32<T>(v[n]); });
                            }
                            mend<T, N>(p, sh, !isfinite(low), n0, min(n0 + 16, m.tokens), col);
                        };
                        put(lo, low_lo, col0 + row);
                        put(hi, low_hi, col0 + kHalfRows + row);
                    }
                }
                fence_before();
                bar_arrive(&sh.acc_empty[b]);
                if (phase == 1) epilogue_sync();                     // chosen and row_weight are the next tile's now
                x = end;
                ++at;
            }
        }
        __syncwarp();
        // every role advances by the same stages and segments
        turn += last - first;
        if (last > first) acc += (last - 1) / split.depth - first / split.depth + 1;
    }

    if (active > 0) {
        grid.sync();
        const uint32_t pairs = (uint32_t)(sh.parted_tiles[1] * m.tokens);
        for (uint32_t u = blockIdx.x * kWarps + warp; u < pairs; u += gridDim.x * kWarps) {
            const uint32_t i = u / (uint32_t)m.tokens;
            const int t = (int)(u - i * (uint32_t)m.tokens), quad = lane * 4;
            const PartedTile part = sh.parted[1][i];
            float4 lo, hi;
            add_parts(p, part.c0, part.c1, t, quad, lo, hi);
            T* y = (T*)m.y + t * m.ld_y;
            const bool bad = __ldcg(p.bad + part.tile) != 0;             // somewhere in the tile
            auto put = [&](const float4& v, int64_t col) {
                store4(y, col, m.hidden, v);
                if (!bad) return;
                const float e[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int j = 0; j < 4; ++j) mend<T, N>(p, sh, !isfinite(e[j]), t, t + 1, col + j);
            };
            put(lo, (int64_t)part.tile * kTileRows + quad);
            put(hi, (int64_t)part.tile * kTileRows + kHalfRows + quad);
        }
    }

    __syncthreads();
    if (sh.fault) {
        // a wait gave up: let what is in flight land before the memory is given
        // back, which for a slot is the last stage that it was armed for
        if (threadIdx.x < kStages && threadIdx.x < sh.armed) {
            const uint32_t turns = (sh.armed - 1 - threadIdx.x) / kStages;
            stage_wait(smem_u32(&sh.full[threadIdx.x]), turns & 1, globaltimer_ns() + kStageWaitNs, kStageWaitNs);
        }
        if (warp == 1 && lane == 0) {
            commit(&sh.drained);
            stage_wait(smem_u32(&sh.drained), 0, globaltimer_ns() + kStageWaitNs, kStageWaitNs);
        }
        __syncthreads();
    }
    if (warp == 1) {
        fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(kTmem) : "memory");
    }
}

// ---- host side --------------------------------------------------------------------

struct TensorPlan {
    size_t logits, act, partial, bad, ids, weights, bytes;
    int64_t most, in_tiles, out_tiles;
};

int padded_tokens(int64_t tokens) { return tokens <= 8 ? 8 : (int)((tokens + 15) / 16 * 16); }

TensorPlan tensor_plan(int64_t tokens, int64_t hidden, int64_t inter, int experts, int top_k)
{
    auto up = [](size_t n) { return (n + 255) / 256 * 256; };
    TensorPlan t;
    t.most = tokens * top_k < experts ? tokens * top_k : experts;
    t.in_tiles = (inter + kHalfRows - 1) / kHalfRows;
    t.out_tiles = (hidden + kTileRows - 1) / kTileRows;
    size_t at = 0;
    t.logits = at, at += up((size_t)tokens * experts * 4);
    t.act = at, at += up((size_t)t.most * 2 * padded_tokens(tokens) * inter * 2);
    t.partial = at, at += up((size_t)2 * kGrid * tokens * kTileRows * 4);
    t.bad = at, at += up((size_t)t.out_tiles * 4);
    t.ids = at, at += up((size_t)tokens * top_k * 4);
    t.weights = at, at += up((size_t)tokens * top_k * 4);
    t.bytes = at;
    return t;
}

// `count` matrices of [rows, cols] elements at pitch ld, one after another;
// boxes of kDepth columns x box_rows rows of one matrix. What lies outside its
// matrix is zeros and is not read.
bool encode_matrices(CUtensorMap* map, const void* base, int64_t count, int64_t rows, int64_t cols, int64_t ld,
                     int box_rows, bool f16)
{
    const TensorMapEncoder enc = tensor_map_encoder();
    if (!enc) return false;
    const cuuint64_t dims[3] = {(cuuint64_t)cols, (cuuint64_t)rows, (cuuint64_t)count};
    const cuuint64_t strides[2] = {(cuuint64_t)ld * 2, (cuuint64_t)ld * 2 * (cuuint64_t)rows};
    const cuuint32_t box[3] = {kDepth, (cuuint32_t)box_rows, 1};
    const cuuint32_t steps[3] = {1, 1, 1};
    return enc(map, f16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3,
               const_cast<void*>(base), dims, strides, box, steps, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <class T, int N>
cudaError_t launch(MoeTensorParams& p, cudaStream_t s)
{
    const size_t smem = kSharedHead + 1024 + (size_t)kRing<N> * kStageBytes<N>;
    const void* kernel = (const void*)moe_tensor_kernel<T, N>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    void* args[] = {(void*)&p};
    const int sms = sm_count();
    return cudaLaunchCooperativeKernel(kernel, dim3((unsigned)(sms < kGrid ? sms : kGrid)), dim3(kThreads), args, smem,
                                       s);
}

template <class T>
cudaError_t launch_for(MoeTensorParams& p, cudaStream_t s)
{
    switch (padded_tokens(p.m.tokens)) {
    case 8: return launch<T, 8>(p, s);
    case 16: return launch<T, 16>(p, s);
    case 32: return launch<T, 32>(p, s);
    case 48: return launch<T, 48>(p, s);
    default: return launch<T, 64>(p, s);
    }
}

}  // namespace

size_t moe_tensor_workspace(int64_t tokens, int64_t hidden, int64_t inter, int experts, int top_k)
{
    return tensor_plan(tokens, hidden, inter, experts, top_k).bytes;
}

bool launch_moe_tensor(const MoeParams& m, int dtype, cudaStream_t s, cudaError_t* e)
{
    const TensorPlan t = tensor_plan(m.tokens, m.hidden, m.inter, m.experts, m.top_k);
    // stages are counted in 32 bits
    if (t.most * t.in_tiles * ((m.hidden + kDepth - 1) / kDepth) > INT32_MAX ||
        t.out_tiles * t.most * ((m.inter + kDepth - 1) / kDepth) > INT32_MAX)
        return false;
    const int n = padded_tokens(m.tokens);
    const bool f16 = dtype == PTOC_F16;
    MoeTensorParams p;
    memset(&p, 0, sizeof(p));
    p.m = m;
    p.logits = (float*)(m.ws + t.logits);
    p.act = m.ws + t.act;
    p.partial = (float*)(m.ws + t.partial);
    p.bad = (uint32_t*)(m.ws + t.bad);
    p.ids = (int32_t*)(m.ws + t.ids);
    p.weights = (float*)(m.ws + t.weights);
    p.wait_ns = copy_wait_ns();
    if (!encode_matrices(&p.w_in, m.w_in, 2 * (int64_t)m.local, m.inter, m.hidden, m.hidden, kHalfRows, f16) ||
        !encode_matrices(&p.w_out, m.w_out, m.local, m.hidden, m.inter, m.inter, kHalfRows, f16) ||
        !encode_matrices(&p.x, m.x, 1, m.tokens, m.hidden, m.tokens > 1 ? m.ld_x : m.hidden, n < 16 ? 16 : n, f16) ||
        !encode_matrices(&p.h, p.act, t.most, 2 * n, m.inter, m.inter, 2 * n, f16))
        return false;
    *e = f16 ? launch_for<__half>(p, s) : launch_for<__nv_bfloat16>(p, s);
    return true;
}

cudaError_t take_stage_faults_moe(uint32_t* count) { return take_stage_faults(count); }

}  // namespace ptoc
