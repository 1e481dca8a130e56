// The products of the gated feed-forward block and of its backward pass on the
// tensor cores: one persistent kernel, whose operands and epilogue follow the
// product (Product, below).
//
//   kIn       [g, u] = x w_in^T        h = act(g) u                  (and pre)
//   kOut      y  = h w_out^T
//   kBackIn   dh = dy w_out            dg = dh u act'(g), du = dh act(g), h = act(g) u
//   kBackX    dx = dg w_gate + du w_up
//   kGrad     the same, d_w_in = [dg, du]^T x and d_w_out = dy^T h (over the tokens), those that are asked for
//
// h, dg and du pass between the products in PARTS numbers of the type: one, rounded as
// a tensor core reads it, or where the caller asks for it two, the second one what
// the first left, as further planes of the contraction. One makes the error of a
// result sqrt(2) times that of its own rounding (2.35e-3 of the norm where that is
// 1.65e-3, bf16); two make the products that read them twice as long (8192 tokens of
// 4096 x 12288 1660 us forward where one takes 1230, 4870 backward where one takes
// 2590; 512 tokens 133 and 99, 331 and 207).
//
// Two SMs (a cluster of two blocks) work on one tile of 256 rows x BN columns:
// each holds 128 rows of A and half of B's columns in shared memory, and the
// mma (cta_group::2, issued by the first block) reads both halves, so that a
// block copies and reads 32 KB per 64 elements of depth where it would need 48
// alone. Copies run through a ring of stages; the accumulators, 128 rows x BN
// columns of each block's tensor memory, are two in turn, so that the epilogue
// of a tile overlaps the next tile's products. In kIn the first block's half of
// B are gate rows and the second's the up rows of the same columns: g and u of an
// element are in the same lane, BN / 2 columns apart.
//
// Operands that lie along the other direction (the contraction over hidden of
// w_out, over inter of w_in, over the tokens of both sides of a weight's gradient) are read
// as they are: boxes of 64 columns x 64 rows, and the descriptor's M- or N-major
// form; nothing is transposed in memory.
//
// Measured on GB300 (bf16; a library's plain product of the same size in
// brackets): 8192 tokens of 4096 x 12288 1230 us forward (1262), 1300 with pre
// kept, 2700 backward (2530), while the clock holds; under the power cap 1440 with
// pre and 2950. Tensor pipes busy (2048 x 4096 x 4096, ncu): kIn 88 %, kOut 83 %,
// kBackIn 67 %, kGrad 94 %. A stage of a tile of 256 columns takes 535 cycles, of
// which the products take 512; narrower tiles are bound by the copies: 310 cycles
// for 128 columns (24 KB to an SM), 260 for 64. A tile's drain takes 3,500 cycles,
// in kBackIn 21,000 (five numbers moved for each element), so that batches with
// hidden below 2,560 are bound by it there. 1003 tokens of 2048 x 5000 105 us backward.
//
// Roles: warp 0 copies A, warp 2 copies B, warp 1 multiplies, warps 4 to 11 drain
// (their quarter of the tensor memory's lanes is warp % 4; the first four take
// the first half of the columns). Tiles go in groups of kGroupRows tile
// rows, so that what the clusters read at a time stays in L2.
#pragma once

#include <cstring>

#include "dense/ffn_act.cuh"
#include "dense/ffn_common.cuh"
#include "dense/ffn_few.cuh"
#include "layers/layers_common.cuh"
#include "layers/tensor_core.cuh"

namespace ptoc {

namespace {

enum Product : int { kIn = 0, kOut = 1, kBackIn = 2, kBackX = 3, kGrad = 4 };

constexpr int kDepth = 64;                  // a stage: 64 elements (128 bytes, one swizzle row) of K
constexpr int kRows = 128;                  // rows of A in a block
constexpr int kDrainWarps = 8;              // two for each quarter of the tensor memory's lanes
constexpr int kThreads = 128 + 32 * kDrainWarps;
constexpr int kGroupRows = 8;
constexpr int kMaxStages = 9;
constexpr int kClusters = 76;               // pairs of SMs
constexpr int kStageCycles = 535;           // of a stage of a tile of 256 columns
constexpr int kDrainCycles = 3500;          // of a tile's drain

// Whether B's rows run along the contraction (K) rather than along it being their
// columns. A's do in the weights' gradients.
template <int PRODUCT>
constexpr bool kBByRows = PRODUCT >= kBackIn;

// A result and its operands.
struct Problem {
    CUtensorMap a, b;
    CUtensorMap out;                        // the result; kIn: h; kBackIn: dg, du and h, its planes (PARTS times)
    int64_t rows, cols;                     // of the result (d_w_in: of one plane)
    uint32_t tiles_m, tiles_n;              // tiles_m: of all planes
    uint32_t plane_tiles;                   // tile rows of a plane
    int32_t depth;                          // stages of one plane of the contraction
};

struct ProductParams {
    Problem q[3];                           // kGrad: dx, d_w_in and d_w_out (tiles 0: not asked for); else the first
    CUtensorMap pre_out;                    // kIn: g and u, its planes
    const void* pre;                        // kBackIn (read); kIn: null where pre is not kept
    int64_t ld_pre, inter;                  // inter: from g to u in a row of pre
    int32_t parts;                          // of what kOut, kBackX and kGrad read
    uint32_t tiles;                         // of all problems
    uint32_t rounds;                        // kGrad: see Order
    uint64_t wait_ns;
};

struct Shared {
    uint64_t full[kMaxStages], empty[kMaxStages];
    uint64_t acc_full[2], acc_empty[2], drained;
    uint32_t tmem;
    int32_t fault;                          // a bounded wait of either block gave up
    uint32_t sent[2];                       // stages whose copies of A and of B this block started
};

constexpr uint32_t kHead = 1024;
constexpr int kChunk = 32;                  // columns that a drain warp handles at a time
constexpr uint32_t kBuffer = 32 * kChunk * 2;
constexpr uint32_t kDrainBytes = kDrainWarps * 2 * kBuffer;
constexpr uint32_t kSharedMost = 227 * 1024;
template <int BN>
constexpr uint32_t kStageBytes = (kRows + BN / 2) * kDepth * 2;
template <int BN>
constexpr int kStages = (int)((kSharedMost - kHead - 1024 - kDrainBytes) / kStageBytes<BN>) < kMaxStages
                            ? (int)((kSharedMost - kHead - 1024 - kDrainBytes) / kStageBytes<BN>)
                            : kMaxStages;
template <int BN>
constexpr uint32_t kSharedBytes = kHead + 1024 + kStages<BN> * kStageBytes<BN> + kDrainBytes;

// ---- instructions of a pair of blocks -------------------------------------------------

// (what it hands over are columns of tensor memory, which the fences order)
__device__ __forceinline__ void remote_arrive(uint32_t bar)
{
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

// Bytes that a barrier of this block waits for, without an arrival; and bytes
// that will not come.
__device__ __forceinline__ void bar_more(uint64_t* bar, uint32_t bytes)
{
    asm volatile("mbarrier.expect_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(bar)), "r"(bytes) : "memory");
}

__device__ __forceinline__ void bar_less(uint64_t* bar, uint32_t bytes)
{
    asm volatile("mbarrier.complete_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(bar)), "r"(bytes)
                 : "memory");
}

// Sixteen columns from `lo_at` and from `hi_at` on of this thread's row of tensor memory.
__device__ __forceinline__ void store_columns(uint32_t lo_at, uint32_t hi_at, const float (&lo)[16], const float (&hi)[16])
{
    auto store = [](uint32_t at, const float (&v)[16]) {
        asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 "
                     "[%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};"
                     ::"r"(at), "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]),
                       "f"(v[8]), "f"(v[9]), "f"(v[10]), "f"(v[11]), "f"(v[12]), "f"(v[13]), "f"(v[14]), "f"(v[15])
                     : "memory");
    };
    store(lo_at, lo);
    store(hi_at, hi);
    asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

__device__ __forceinline__ void remote_write(uint32_t addr, uint32_t v)
{
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

// A box into this block's memory, which completes on a barrier of either block.
__device__ __forceinline__ void pair_copy(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint32_t bar)
{
    asm volatile("cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
                 "[%0], [%1, {%2, %3, %4}], [%5];"
                 ::"r"(dst), "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar)
                 : "memory");
}

__device__ __forceinline__ void pair_mma(uint32_t d, uint64_t a, uint64_t b, uint32_t kind, uint32_t accumulate)
{
    asm volatile("{ .reg .pred p; setp.ne.u32 p, %4, 0;\n"
                 "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p; }"
                 ::"r"(d), "l"(a), "l"(b), "r"(kind), "r"(accumulate)
                 : "memory");
}

// The barrier of both blocks completes when every mma issued so far by this thread has.
__device__ __forceinline__ void pair_commit(uint64_t* bar)
{
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;"
                 ::"r"(smem_u32(bar)), "h"((uint16_t)3)
                 : "memory");
}

// A bounded wait on a barrier of this block; a role whose wait gave up ends, so
// that no barrier sees a phase that its other side did not.
__device__ __forceinline__ bool wait(Shared& sh, uint64_t* bar, uint32_t parity, uint64_t bound_ns)
{
    if (bounded_wait(smem_u32(bar), parity, bound_ns, &sh.fault)) return true;
    if (atomicExch(&sh.fault, 1) == 0) atomicAdd(&g_stage_faults, 1u);
    remote_write(in_block(smem_u32(&sh.fault), cluster_rank() ^ 1), 1);
    return false;
}

// ---- tiles ----------------------------------------------------------------------------

// The tiles of a cluster, in turn. In kGrad dx's tiles, which are deep (twice
// inter), come first, and the clusters that take one more of them than the others
// join the weights' tiles later, by as many rounds as fit into one of dx's: a last
// wave of a few deep tiles leaves no cluster idle. Clusters that work at the same
// time work on neighbouring tiles.
template <int PRODUCT>
struct Order {
    uint32_t cluster, clusters, deep, more, tiles;           // deep: this cluster's tiles of dx; more: clusters with one more
    uint32_t first;                                          // of the weights' tiles
    __device__ __forceinline__ Order(const ProductParams& p)
        : cluster(blockIdx.x >> 1), clusters(gridDim.x >> 1), deep(0), more(0), tiles(p.tiles), first(0)
    {
        if (PRODUCT == kGrad) {
            first = p.q[0].tiles_m * p.q[0].tiles_n;
            deep = first / clusters;
            more = first - deep * clusters;
            if (cluster < more) ++deep;
        }
    }
    // The cluster's tile k; false if there is none.
    __device__ __forceinline__ bool tile(const ProductParams& p, uint32_t k, uint32_t& t) const
    {
        if (PRODUCT != kGrad || k < deep) {
            t = cluster + k * clusters;
            return t < tiles;
        }
        const uint32_t j = k - deep, others = clusters - more;
        if (cluster < more) t = p.rounds * others + j * clusters + cluster;
        else if (j < p.rounds) t = j * others + (cluster - more);
        else t = p.rounds * others + (j - p.rounds) * clusters + cluster;
        t += first;
        return t < tiles;
    }
};

// (In 32 bits: the limits of the sizes keep them below. Three divisions in 64 for
// every tile took longer than a short tile's products.)
template <int PRODUCT>
struct Tile {
    uint32_t m, n, plane, which;            // in tiles; m within its plane; the problem
    __device__ __forceinline__ Tile(const ProductParams& p, uint32_t t) : which(0)
    {
        if (PRODUCT == kGrad)
            for (; which < 2; ++which) {
                const uint32_t here = p.q[which].tiles_m * p.q[which].tiles_n;
                if (t < here) break;
                t -= here;
            }
        const Problem& q = p.q[which];
        const uint32_t group = kGroupRows * q.tiles_n, g = t / group, at = t - g * group;
        const uint32_t rows = min((uint32_t)kGroupRows, q.tiles_m - g * kGroupRows);
        n = rows == kGroupRows ? at / kGroupRows : at / rows;
        m = g * kGroupRows + (at - n * rows);
        plane = m >= q.plane_tiles;         // (there are two at most)
        m -= plane * q.plane_tiles;
    }
    // The stages of a tile of a problem: of the planes of its contraction, which are
    // dg and du in dx, and the parts.
    static __host__ __device__ __forceinline__ uint32_t stages(uint32_t depth, uint32_t parts, uint32_t which)
    {
        const bool two = PRODUCT == kBackX || (PRODUCT == kGrad && which == 0);
        return depth * (PRODUCT == kIn || PRODUCT == kBackIn ? 1u : two ? 2 * parts : parts);
    }
    static __device__ __forceinline__ uint32_t stages(const ProductParams& p, uint32_t which)
    {
        return stages((uint32_t)p.q[which].depth, (uint32_t)p.parts, which);
    }
    // The planes of A and of B in plane n of the contraction. (What has parts lies
    // as dg, du, h and then their second parts.)
    __device__ __forceinline__ int plane_a(int n) const
    {
        if (PRODUCT == kOut) return n;
        if (PRODUCT == kBackX || (PRODUCT == kGrad && which == 0)) return n + (n >> 1);
        return PRODUCT == kGrad && which == 1 ? (int)plane + 3 * n : 0;
    }
    __device__ __forceinline__ int plane_b(int n) const
    {
        if (PRODUCT == kBackX || (PRODUCT == kGrad && which == 0)) return n & 1;
        return PRODUCT == kGrad && which == 2 ? 3 * n : 0;
    }
};

// The sums of a tile deeper than kChain stages are taken at every chain's end and added up in
// the other accumulator's columns (its drains are then not hidden: about 1 % of its time).
// Where a tile's sums stand: which accumulator, and how often each was used before.
// Tiles take the two in turn; a deep one takes the first for all its chains (its sums so far
// are in the second), and so does the tile after it, which waits until both are read.
// DEEP: there are such tiles. (The same for all: dx and the weights' gradients of 512 tokens
// of 4096 x 12288 209 us instead of 205.)
template <bool DEEP>
struct Turn {
    uint32_t b = 0, used[2] = {0, 0};
    static __device__ __forceinline__ uint32_t chains(uint32_t stages)
    {
        return DEEP ? (stages + (uint32_t)kChain - 1) / (uint32_t)kChain : 1u;
    }
    __device__ __forceinline__ void begin(uint32_t chains) { b = DEEP && chains > 1 ? 0 : b; }
    __device__ __forceinline__ uint32_t phase() const { return (b ? used[1] : used[0]) & 1; }
    __device__ __forceinline__ void next() { ++(b ? used[1] : used[0]); }
    __device__ __forceinline__ void end(uint32_t chains) { b = DEEP && chains > 1 ? 0 : b ^ 1; }
};

// Eight neighbouring elements.
template <class T>
__device__ __forceinline__ uint4 pack8(const float* v)
{
    return make_uint4(pack2<T>(pair(v[0], v[1])), pack2<T>(pair(v[2], v[3])), pack2<T>(pair(v[4], v[5])),
                      pack2<T>(pair(v[6], v[7])));
}

template <class T>
__device__ __forceinline__ void unpack8(const uint4& w, float* v)
{
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
        v[2 * i] = Raw8<T, 8>::widen(u[i] & 0xffffu), v[2 * i + 1] = Raw8<T, 8>::widen_high(u[i]);
}

// What eight elements leave of the values they stand for, rounded (nothing of one
// that is not finite): f16 in steps of 2^-24 at the least.
template <class T>
__device__ __forceinline__ uint4 rest8(const float* v, const uint4& w)
{
    float high[8], rest[8];
    unpack8<T>(w, high);
#pragma unroll
    for (int i = 0; i < 8; ++i) rest[i] = v[i] - high[i], rest[i] = isfinite(rest[i]) ? rest[i] : 0.0f;
    return pack8<T>(rest);
}

// A drain warp's two buffers of 32 rows x 32 columns, a row to a lane, in the
// 64-byte swizzle (16-byte words of a row exchanged by bits 1 and 2 of the row,
// so that eight lanes touch all banks). Results leave as boxes of a tensor map,
// which clips them: stored by the lanes, 16 bytes to a row, they kept the copies
// of the products waiting (8192 x 4096 x 12288: dh 957 us, where the product
// alone takes 413).
struct DrainBuffers {
    uint32_t base, lane;
    int turn = 0;

    __device__ __forceinline__ uint32_t word(uint32_t buffer, uint32_t row, uint32_t w) const
    {
        return base + buffer * kBuffer + row * (kChunk * 2) + (w ^ (row >> 1 & 3)) * 16;
    }
    // Until at most `left` boxes still have to be read from the buffers.
    template <int LEFT>
    __device__ __forceinline__ void wait_read() const
    {
        if (lane == 0) asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(LEFT) : "memory");
        __syncwarp();
    }
    // Store this lane's row of 32 columns as a part of the box at column x, row y, plane z.
    __device__ __forceinline__ void put(const uint4 (&w)[4], const CUtensorMap* map, int x, int y, int z)
    {
        wait_read<1>();
#pragma unroll
        for (uint32_t i = 0; i < 4; ++i)
            asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};"
                         ::"r"(word(turn, lane, i)), "r"(w[i].x), "r"(w[i].y), "r"(w[i].z), "r"(w[i].w) : "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) {
            asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%1, %2, %3}], [%4];"
                         ::"l"(map), "r"(x), "r"(y), "r"(z), "r"(base + turn * kBuffer) : "memory");
            asm volatile("cp.async.bulk.commit_group;" ::: "memory");
        }
        turn ^= 1;
    }
    // Start copying 32 rows x 32 columns of g and of u into the two buffers.
    template <class T>
    __device__ __forceinline__ void fetch(const ProductParams& p, int64_t row0, int64_t col0) const
    {
        wait_read<0>();
        if (row0 < p.q[0].rows && col0 < p.q[0].cols) {
            const uint32_t w = lane & 3;
#pragma unroll
            for (uint32_t i = 0; i < 4; ++i) {
                const uint32_t r = i * 8 + (lane >> 2);
                const T* from = (const T*)p.pre + (row0 + r) * p.ld_pre + col0 + w * 8;
                if (row0 + r < p.q[0].rows && col0 + w * 8 < p.q[0].cols)
#pragma unroll
                    for (uint32_t b = 0; b < 2; ++b)
                        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;"
                                     ::"r"(word(b, r, w)), "l"(from + b * p.inter) : "memory");
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    }
    __device__ __forceinline__ void fetched() const
    {
        asm volatile("cp.async.wait_group 0;" ::: "memory");
        __syncwarp();
    }
    // Word w of this lane's row.
    __device__ __forceinline__ uint4 get(uint32_t buffer, uint32_t w) const
    {
        uint4 v;
        asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(word(buffer, lane, w)) : "memory");
        return v;
    }
};

// Sixteen columns of an accumulator from `lo_at` and from `hi_at` on; more: and what
// earlier chains of the tile left, BN columns further on.
template <int BN, bool DEEP>
__device__ __forceinline__ void load_sums(uint32_t lo_at, uint32_t hi_at, bool more, float (&lo)[16], float (&hi)[16])
{
    load_columns(lo_at, hi_at, lo, hi);
    if (!DEEP || !more) return;
    float a[16], b[16];
    load_columns(lo_at + BN, hi_at + BN, a, b);
#pragma unroll
    for (int i = 0; i < 16; ++i) lo[i] += a[i], hi[i] += b[i];
}

// A chain's sums of a warp's part of a tile, to those of the chains before it.
template <int PRODUCT, int BN>
__device__ __forceinline__ void keep_sums(uint32_t acc, bool more)
{
    constexpr int kColumns = PRODUCT == kIn ? BN / 4 : BN / 2, kStep = PRODUCT == kIn ? 16 : 32;
#pragma unroll 1
    for (int c = 0; c < kColumns; c += kStep) {
        const uint32_t lo_at = acc + c, hi_at = lo_at + (PRODUCT == kIn ? BN / 2 : 16);
        float lo[16], hi[16];
        load_sums<BN, true>(lo_at, hi_at, more, lo, hi);
        store_columns(lo_at + BN, hi_at + BN, lo, hi);
    }
}

// A warp's part of a tile: rows row0 to row0 + 31 (of plane `plane`), the
// accumulator's columns from `acc` on, which are the result's from col0 on. more: see load_sums.
template <class T, int PRODUCT, int ACT, int BN, int PARTS, bool DEEP>
__device__ __forceinline__ void drain(const ProductParams& p, DrainBuffers& buf, uint32_t acc, bool more, int64_t row0,
                                      int64_t plane, int64_t col0, const Problem& q)
{
    if (row0 >= q.rows) return;
    constexpr int kColumns = PRODUCT == kIn ? BN / 4 : BN / 2;
#pragma unroll 1
    for (int c = 0; c < kColumns; c += kChunk) {
        if (col0 + c >= q.cols) break;
        const int x = (int)(col0 + c), y = (int)row0;
        if constexpr (PRODUCT == kIn) {
            uint4 h[4], rest[4], g[4], u[4];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                float vg[16], vu[16], vh[16];
                load_sums<BN, DEEP>(acc + c + 16 * k, acc + BN / 2 + c + 16 * k, more, vg, vu);
#pragma unroll
                for (int i = 0; i < 16; ++i) vh[i] = act_value<ACT>(vg[i]) * vu[i];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    h[2 * k + i] = pack8<T>(vh + 8 * i);
                    if constexpr (PARTS == 2) rest[2 * k + i] = rest8<T>(vh + 8 * i, h[2 * k + i]);
                    g[2 * k + i] = pack8<T>(vg + 8 * i);
                    u[2 * k + i] = pack8<T>(vu + 8 * i);
                }
            }
            buf.put(h, &q.out, x, y, 0);
            if constexpr (PARTS == 2) buf.put(rest, &q.out, x, y, 1);
            if (p.pre) {
                buf.put(g, &p.pre_out, x, y, 0);
                buf.put(u, &p.pre_out, x, y, 1);
            }
        } else if constexpr (PRODUCT == kBackIn) {
            // (the first chunk's g and u are on their way already)
            float dh[32];
            load_sums<BN, DEEP>(acc + c, acc + c + 16, more, *(float(*)[16])dh, *(float(*)[16])(dh + 16));
            buf.fetched();
            if constexpr (PARTS == 1) {
                uint4 dg[4], du[4], h[4];
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    float g[8], u[8], vg[8], vu[8], vh[8];
                    unpack8<T>(buf.get(0, w), g);
                    unpack8<T>(buf.get(1, w), u);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float d = dh[8 * w + i];
                        const Act a = act_both<ACT>(g[i]);
                        vg[i] = d * u[i] * a.slope;
                        vu[i] = d * a.value;
                        vh[i] = a.value * u[i];
                    }
                    dg[w] = pack8<T>(vg), du[w] = pack8<T>(vu), h[w] = pack8<T>(vh);
                }
                __syncwarp();
                buf.put(dg, &q.out, x, y, 0);
                buf.put(du, &q.out, x, y, 1);
                buf.put(h, &q.out, x, y, 2);
            } else {
                // one result at a time: six of them do not fit into registers
                uint4 wg[4], wu[4];
#pragma unroll
                for (int w = 0; w < 4; ++w) wg[w] = buf.get(0, w), wu[w] = buf.get(1, w);
                __syncwarp();
#pragma unroll 1
                for (int r = 0; r < 3; ++r) {
                    uint4 high[4], rest[4];
#pragma unroll
                    for (int w = 0; w < 4; ++w) {
                        float g[8], u[8], v[8];
                        unpack8<T>(wg[w], g);
                        unpack8<T>(wu[w], u);
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const float d = dh[8 * w + i];
                            const Act a = act_both<ACT>(g[i]);
                            v[i] = r == 0 ? d * u[i] * a.slope : r == 1 ? d * a.value : a.value * u[i];
                        }
                        high[w] = pack8<T>(v);
                        rest[w] = rest8<T>(v, high[w]);
                    }
                    buf.put(high, &q.out, x, y, r);
                    buf.put(rest, &q.out, x, y, 3 + r);
                }
            }
            if (c + kChunk < kColumns) buf.template fetch<T>(p, row0, col0 + c + kChunk);
        } else {
            float v[32];
            load_sums<BN, DEEP>(acc + c, acc + c + 16, more, *(float(*)[16])v, *(float(*)[16])(v + 16));
            uint4 w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = pack8<T>(v + 8 * i);
            buf.put(w, &q.out, x, y, (int)plane);
        }
    }
}

template <class T, int PRODUCT, int ACT, int BN, int PARTS, bool DEEP>
__global__ void __launch_bounds__(kThreads, 1) ffn_product_kernel(const __grid_constant__ ProductParams p)
{
    extern __shared__ unsigned char raw[];
    Shared& sh = *(Shared*)raw;
    constexpr uint32_t kRing = kStages<BN>, kStage = kStageBytes<BN>, kABytes = kRows * kDepth * 2;
    constexpr uint32_t kTmem = 2 * BN;
    constexpr bool kB = kBByRows<PRODUCT>;
    // f32 accumulator, both operands T, 256 rows, BN columns
    constexpr uint32_t kType = std::is_same<T, __half>::value ? 0u : 1u;
    constexpr uint32_t kKind = 1u << 4 | kType << 7 | kType << 10 | (uint32_t)kB << 16 |
                               (uint32_t)(BN >> 3) << 17 | (uint32_t)(2 * kRows >> 4) << 24;
    const uint32_t ring = (smem_u32(raw) + kHead + 1023u) & ~1023u;
    const int lane = threadIdx.x & 31, warp = uniform_warp();
    const uint32_t rank = cluster_rank();
    const Order<PRODUCT> order(p);

    if (threadIdx.x == 0) {
        for (uint32_t s = 0; s < kRing; ++s) bar_init(&sh.full[s], 1), bar_init(&sh.empty[s], 1);
        for (int b = 0; b < 2; ++b) bar_init(&sh.acc_full[b], 1), bar_init(&sh.acc_empty[b], 2 * kDrainWarps);
        bar_init(&sh.drained, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        sh.fault = 0;
        sh.sent[0] = sh.sent[1] = 0;
        if (PRODUCT != kGrad || p.q[0].tiles_m) prefetch_map(&p.q[0].a), prefetch_map(&p.q[0].b);
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&sh.tmem)),
                     "n"(kTmem)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
        fence_before();
    }
    __syncthreads();
    cluster_sync();                         // the other block's barriers are there too
    fence_after();
    const uint32_t tmem = sh.tmem;
    pdl_enter();

    if (warp == 0 || warp == 2) {
        // what an earlier launch stored (h, dg, du) is read by the copies
        asm volatile("fence.proxy.async;" ::: "memory");
        const uint32_t full = in_block(smem_u32(&sh.full[0]), 0);        // the first block's barriers
        uint32_t u = 0, slot = 0, turn = 1, t;
        bool ok = true;
        for (uint32_t i = 0; ok && order.tile(p, i, t); ++i) {
            const Tile<PRODUCT> tile(p, t);
            const Problem& q = p.q[PRODUCT == kGrad ? tile.which : 0];
            const bool by_rows = PRODUCT == kGrad && tile.which > 0;
            const uint32_t stages = tile.stages(p, PRODUCT == kGrad ? tile.which : 0);
            const int m0 = (int)(tile.m * 2 * kRows + rank * kRows);
            const int n0 = PRODUCT == kIn ? (int)tile.n * (BN / 2) : (int)tile.n * BN + (int)rank * (BN / 2);
            int k = 0, plane = 0;
            for (uint32_t it = 0; it < stages; ++it, ++u) {
                ok = __all_sync(0xffffffffu, wait(sh, &sh.empty[slot], turn, p.wait_ns));
                if (!ok) break;
                const uint32_t bar = full + slot * 8, at = ring + slot * kStage;
                if (elect_one()) {
                    if (warp == 0) {
                        // the first block expects the bytes of both
                        if (rank == 0) bar_expect(&sh.full[slot], 2 * kStage);
                        if (by_rows) {
                            pair_copy(at, &q.a, m0, k, tile.plane_a(plane), bar);
                            pair_copy(at + kABytes / 2, &q.a, m0 + 64, k, tile.plane_a(plane), bar);
                        } else {
                            pair_copy(at, &q.a, k, m0, tile.plane_a(plane), bar);
                        }
                    } else if constexpr (kB) {
#pragma unroll
                        for (int c = 0; c < BN / 2; c += 64)
                            pair_copy(at + kABytes + c * 128, &q.b, n0 + c, k, tile.plane_b(plane), bar);
                    } else {
                        pair_copy(at + kABytes, &q.b, k, n0, PRODUCT == kIn ? (int)rank : 0, bar);
                    }
                }
                __syncwarp();
                if (++slot == kRing) slot = 0, turn ^= 1;
                k += kDepth;
                if (PRODUCT != kIn && PRODUCT != kBackIn && k >= q.depth * kDepth) k = 0, ++plane;
            }
        }
        if (lane == 0) sh.sent[warp >> 1] = u;
        // the last arrivals at the barriers of this block
        for (uint32_t i = 0; i < kRing && i < u && ok; ++i) {
            const uint32_t v = u - 1 - i;
            ok = __all_sync(0xffffffffu, wait(sh, &sh.empty[v % kRing], v / kRing & 1, p.wait_ns));
        }
    }

    if (warp == 1 && rank == 0) {
        uint32_t slot = 0, turn = 0, t;
        bool ok = true, ready = false;      // ready: the next stage is known to have landed
        Turn<DEEP> acc;
        const uint64_t desc_b = operand_at<kB>(ring + kABytes, 0);
        for (uint32_t i = 0; ok && order.tile(p, i, t); ++i) {
            const uint32_t which = PRODUCT == kGrad ? Tile<PRODUCT>(p, t).which : 0;
            const bool by_rows = PRODUCT == kGrad && which > 0;
            const uint32_t stages = Tile<PRODUCT>::stages(p, which);
            const uint64_t desc_a = by_rows ? operand_by_rows(ring) : operand(ring);
            const uint32_t step_a = (by_rows ? 2048 : 32) >> 4, kind = kKind | (uint32_t)by_rows << 15;
            const uint32_t chains = acc.chains(stages);
            acc.begin(chains);
            for (uint32_t it = 0; ok && it < stages; acc.next()) {
                const uint32_t d = tmem + acc.b * BN, chain = DEEP ? min(stages - it, (uint32_t)kChain) : stages;
                ok = __all_sync(0xffffffffu, wait(sh, &sh.acc_empty[acc.b], acc.phase() ^ 1, p.wait_ns));
                if (!ok) break;
                fence_after();
                for (uint32_t j = 0; j < chain; ++j, ++it) {
                    if (!ready) {
                        ok = __all_sync(0xffffffffu, wait(sh, &sh.full[slot], turn, p.wait_ns));
                        if (!ok) break;
                    }
                    fence_after();
                    const uint64_t a = desc_a + slot * (kStage >> 4), w = desc_b + slot * (kStage >> 4);
                    if (elect_one()) {
#pragma unroll
                        for (int k = 0; k < kDepth / 16; ++k)
                            pair_mma(d, a + k * step_a, w + k * ((kB ? 2048 : 32) >> 4), kind, j > 0 || k > 0);
                        pair_commit(&sh.empty[slot]);
                    }
                    __syncwarp();
                    if (++slot == kRing) slot = 0, turn ^= 1;
                    // asked while the products queue up: a wait after them takes longer than the queue lasts
                    ready = __all_sync(0xffffffffu, landed(smem_u32(&sh.full[slot]), turn));
                }
                if (ok && elect_one()) pair_commit(&sh.acc_full[acc.b]);
                __syncwarp();
            }
            acc.end(chains);
        }
    }

    if (warp >= 4) {
        uint32_t t;
        bool ok = true;
        Turn<DEEP> acc;
        const int half = (warp - 4) >> 2;
        DrainBuffers buf{ring + kRing * kStage + (uint32_t)(warp - 4) * 2 * kBuffer, (uint32_t)lane};
        for (uint32_t i = 0; ok && order.tile(p, i, t); ++i) {
            const Tile<PRODUCT> tile(p, t);
            const Problem& q = p.q[PRODUCT == kGrad ? tile.which : 0];
            const int64_t row0 = (int64_t)tile.m * 2 * kRows + rank * kRows + (warp & 3) * 32;
            constexpr int kHalf = PRODUCT == kIn ? BN / 4 : BN / 2;
            const int64_t col0 = (int64_t)tile.n * 2 * kHalf + half * kHalf;
            const uint32_t chains = acc.chains(DEEP ? tile.stages(p, PRODUCT == kGrad ? tile.which : 0) : 0);
            if constexpr (PRODUCT == kBackIn) buf.template fetch<T>(p, row0, col0);
            acc.begin(chains);
            for (uint32_t k = 0; k < chains; ++k, acc.next()) {
                ok = __all_sync(0xffffffffu, wait(sh, &sh.acc_full[acc.b], acc.phase(), p.wait_ns));
                if (!ok) break;
                __syncwarp();
                fence_after();
                const uint32_t at = tmem + acc.b * BN + ((uint32_t)(warp & 3) << 21) + half * kHalf;
                if (k + 1 < chains) {
                    if constexpr (DEEP) keep_sums<PRODUCT, BN>(at, k > 0);
                } else {
                    drain<T, PRODUCT, ACT, BN, PARTS, DEEP>(p, buf, at, k > 0, row0, tile.plane, col0, q);
                }
                __syncwarp();
                fence_before();
                if (lane == 0) remote_arrive(in_block(smem_u32(&sh.acc_empty[acc.b]), 0));
            }
            acc.end(chains);
        }
        if constexpr (PRODUCT == kBackIn) buf.fetched();
        if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    }

    __syncwarp();
    __syncthreads();
    cluster_sync();                         // neither block starts anything any more
    if (sh.fault || remote_read(in_block(smem_u32(&sh.fault), rank ^ 1))) {
        // A wait gave up: let what is in flight land before the memory is given
        // back. What a stage's barrier expects is brought in line with the copies
        // that were started; of a slot, the last stage tells.
        if (warp == 1 && elect_one()) {     // (the lane that issued the products)
            if (rank == 0) {
                const uint32_t other = in_block(smem_u32(&sh.sent[0]), 1);
                const uint32_t sent[4] = {sh.sent[0], sh.sent[1], remote_read(other), remote_read(other + 4)};
                const uint32_t least = min(min(sent[0], sent[1]), min(sent[2], sent[3]));
                const uint32_t all = max(max(sent[0], sent[1]), max(sent[2], sent[3]));
                for (uint32_t u = least; u < all; ++u) {
                    uint64_t* bar = &sh.full[u % kRing];
                    uint32_t come = 0;
                    for (int i = 0; i < 4; ++i)
                        if (u < sent[i]) come += i & 1 ? kStage - kABytes : kABytes;
                    if (u < sent[0]) bar_less(bar, 2 * kStage - come);
                    else bar_more(bar, come), bar_arrive(bar);
                }
                for (uint32_t i = 0; i < kRing && i < all; ++i) {
                    const uint32_t v = all - 1 - i;
                    stage_wait(smem_u32(&sh.full[v % kRing]), v / kRing & 1, globaltimer_ns() + kStageWaitNs,
                               kStageWaitNs);
                }
                pair_commit(&sh.drained);
            }
            stage_wait(smem_u32(&sh.drained), 0, globaltimer_ns() + kStageWaitNs, kStageWaitNs);
        }
        __syncwarp();
        __syncthreads();
        cluster_sync();
    }
    if (warp == 1) {
        fence_after();
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(kTmem) : "memory");
    }
    cluster_sync();
}

// ---- host side ------------------------------------------------------------------------

template <class T, int PRODUCT, int ACT, int BN, int PARTS, bool DEEP>
cudaError_t launch_tiles(ProductParams& p, cudaStream_t s)
{
    // (at most 2^14 x 2^12 to a problem: the limits of the sizes)
    p.tiles = 0;
    for (const Problem& q : p.q) p.tiles += q.tiles_m * q.tiles_n;
    const int64_t tiles = p.tiles;
    auto kernel = ffn_product_kernel<T, PRODUCT, ACT, BN, PARTS, DEEP>;
    static std::atomic<uint64_t> done{0};
    const int most = sm_count() / 2 < kClusters ? sm_count() / 2 : kClusters;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2 * (unsigned)(tiles < most ? tiles : most));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSharedBytes<BN>;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2, attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = programmatic_launch() ? 2 : 1;
    return launch_shared((const void*)kernel, (int)kSharedBytes<BN>, done,
                         [&] { return cudaLaunchKernelEx(&cfg, kernel, p); });
}

template <int PRODUCT>
bool deep(const ProductParams& p)
{
    for (uint32_t i = 0; i < 3; ++i)
        if (p.q[i].tiles_m && Tile<PRODUCT>::stages((uint32_t)p.q[i].depth, (uint32_t)p.parts, i) > kChain) return true;
    return false;
}

// (deep tiles are always of 256 columns)
template <class T, int PRODUCT, int ACT, int BN, int PARTS>
cudaError_t launch_product(ProductParams& p, cudaStream_t s)
{
    if constexpr (BN == 256)
        if (deep<PRODUCT>(p)) return launch_tiles<T, PRODUCT, ACT, BN, PARTS, true>(p, s);
    return launch_tiles<T, PRODUCT, ACT, BN, PARTS, false>(p, s);
}

// A matrix as an operand or a result: `planes` of [rows, cols], `plane` elements apart.
struct Matrix {
    const void* base;
    int64_t planes, rows, cols, ld, plane;
};

inline Matrix stacked(const void* base, int64_t planes, int64_t rows, int64_t cols, int64_t ld)
{
    return Matrix{base, planes, rows, cols, ld, rows * ld};
}

// (a single row may have any pitch)
template <class T>
bool encode(CUtensorMap* map, const Matrix& m, int box_cols, int box_rows)
{
    const int64_t ld = m.rows > 1 ? m.ld : (m.cols + 7) / 8 * 8;
    return encode_planes(map, m.base, m.planes, m.rows, m.cols, ld, m.planes > 1 ? m.plane : ld * m.rows, box_cols,
                         box_rows, std::is_same<T, __half>::value);
}

// out = a b: A's rows are the result's, or (a_by_rows) both have the tokens as rows.
// out_planes: of which the result's tiles are a plane's each.
template <class T, int PRODUCT, int BN>
bool add_problem(ProductParams& p, int which, const Matrix& a, const Matrix& b, const Matrix& out,
                 bool a_by_rows = false, int out_planes = 1)
{
    const int64_t depth = a_by_rows ? a.rows : a.cols;
    const int64_t columns = PRODUCT == kIn ? BN / 2 : BN;
    Problem& q = p.q[which];
    q.rows = out.rows;
    q.cols = out.cols;
    q.plane_tiles = (uint32_t)((q.rows + 2 * kRows - 1) / (2 * kRows));
    q.tiles_m = q.plane_tiles * (uint32_t)out_planes;
    q.tiles_n = (uint32_t)((q.cols + columns - 1) / columns);
    q.depth = (int32_t)((depth + kDepth - 1) / kDepth);
    p.wait_ns = copy_wait_ns();
    return encode<T>(&q.a, a, 64, a_by_rows ? kDepth : kRows) &&
           encode<T>(&q.b, b, 64, kBByRows<PRODUCT> ? kDepth : BN / 2) && encode<T>(&q.out, out, kChunk, 32);
}

template <class T, int PRODUCT, int ACT, int BN, int PARTS>
cudaError_t product_of(ProductParams& p, const Matrix& a, const Matrix& b, const Matrix& out, cudaStream_t s)
{
    if (!add_problem<T, PRODUCT, BN>(p, 0, a, b, out)) return cudaErrorNotSupported;
    if (PRODUCT == kIn && p.pre) {
        const Matrix pre{p.pre, 2, out.rows, out.cols, p.ld_pre, p.inter};
        if (!encode<T>(&p.pre_out, pre, kChunk, 32)) return cudaErrorNotSupported;
    }
    return launch_product<T, PRODUCT, ACT, BN, PARTS>(p, s);
}

// The width of the tiles: the one with the least waves of clusters times cycles
// of a stage, which were measured (narrower tiles have more bytes to copy for a
// product): 1500 x 7168 x 2048 96 us for h and y in 3 waves of 128 columns, 106 in
// 2 of 256; 2048 x 4096 x 12288 338 in 11 of 256, 360 in 21 of 128.
template <class T, int PRODUCT, int ACT, int PARTS>
cudaError_t product(ProductParams& p, const Matrix& a, const Matrix& b, const Matrix& out, cudaStream_t s)
{
    const int64_t rows = (out.rows + 2 * kRows - 1) / (2 * kRows);
    auto cost = [&](int64_t columns, int64_t cycles) {
        if (PRODUCT == kIn) columns /= 2;
        const int64_t tiles = rows * ((out.cols + columns - 1) / columns);
        return (tiles + kClusters - 1) / kClusters * cycles;
    };
    if (Tile<PRODUCT>::stages((uint32_t)((a.cols + kDepth - 1) / kDepth), (uint32_t)p.parts, 0) > kChain)
        return product_of<T, PRODUCT, ACT, 256, PARTS>(p, a, b, out, s);
    const int64_t wide = cost(256, kStageCycles), middle = cost(128, 310), narrow = cost(64, 260);
    if constexpr (PRODUCT == kOut)
        if (narrow < middle && narrow < wide) return product_of<T, PRODUCT, ACT, 64, PARTS>(p, a, b, out, s);
    if (middle < wide) return product_of<T, PRODUCT, ACT, 128, PARTS>(p, a, b, out, s);
    return product_of<T, PRODUCT, ACT, 256, PARTS>(p, a, b, out, s);
}

template <class T, int ACT, int PARTS>
cudaError_t forward(const FfnParams& q, cudaStream_t s)
{
    const Matrix x = stacked(q.x, 1, q.tokens, q.hidden, q.ld_x);
    const Matrix h = stacked(q.ws, PARTS, q.tokens, q.inter, padded_inter(q.inter));
    const Matrix y = stacked(q.y, 1, q.tokens, q.hidden, q.ld_y);
    const Matrix w_in = stacked(q.w_in, 2, q.inter, q.hidden, q.ld_in);
    const Matrix w_out = stacked(q.w_out, 1, q.hidden, q.inter, q.ld_out);
    ProductParams p;
    memset(&p, 0, sizeof(p));
    p.pre = q.pre, p.ld_pre = q.ld_pre;
    p.inter = q.inter;
    p.parts = PARTS;
    const cudaError_t e = product<T, kIn, ACT, PARTS>(p, x, w_in, h, s);
    return e == cudaSuccess ? product<T, kOut, 0, 1>(p, h, w_out, y, s) : e;
}

template <class T, int ACT, int PARTS>
cudaError_t backward(const FfnBackParams& q, cudaStream_t s)
{
    // with two parts the weights' gradients read both, which few:: does not keep
    const bool streamed = PARTS == 1 && q.tokens <= kFewTokens;
    const BackLayout l = PARTS == 1 ? back_layout(q.tokens, q.inter) : parts_layout(q.tokens, q.inter);
    T* d = (T*)q.ws;
    const Matrix x = stacked(q.x, 1, q.tokens, q.hidden, q.ld_x), dy = stacked(q.dy, 1, q.tokens, q.hidden, q.ld_dy);
    // two parts: dg, du, h and then their second parts, seen as planes from dg and from h on
    const Matrix d_gu{d, PARTS == 1 ? 2 : 5, q.tokens, q.inter, l.ld, l.plane};
    const Matrix h{d + l.h, PARTS == 1 ? 1 : 4, q.tokens, q.inter, l.ld, l.plane};
    ProductParams p;
    memset(&p, 0, sizeof(p));
    p.parts = PARTS;
    cudaError_t e;
    const Matrix w_in = stacked(q.w_in, 2, q.inter, q.hidden, q.ld_in);
    const Matrix d_x = stacked(q.dx, 1, q.tokens, q.hidden, q.ld_dx);
    if (streamed) {
        e = few::backward<T, ACT>(q, s);
    } else {
        const Matrix w_out = stacked(q.w_out, 1, q.hidden, q.inter, q.ld_out);
        p.pre = q.pre, p.ld_pre = q.ld_pre;
        p.inter = q.inter;
        e = product<T, kBackIn, ACT, PARTS>(p, dy, w_out, stacked(d, 3 * PARTS, q.tokens, q.inter, l.ld), s);
        if (e == cudaSuccess && q.dx && !q.d_in && !q.d_out)
            e = product<T, kBackX, 0, 1>(p, d_gu, w_in, d_x, s);
    }
    if (e != cudaSuccess || (!q.d_in && !q.d_out)) return e;
    memset(&p, 0, sizeof(p));
    p.parts = PARTS;
    const Matrix d_in = stacked(q.d_in, 2, q.inter, q.hidden, q.ld_din);
    const Matrix d_out = stacked(q.d_out, 1, q.hidden, q.inter, q.ld_dout);
    if ((q.dx && !streamed && !add_problem<T, kGrad, 256>(p, 0, d_gu, w_in, d_x)) ||
        (q.d_in && !add_problem<T, kGrad, 256>(p, 1, d_gu, x, d_in, true, 2)) ||
        (q.d_out && !add_problem<T, kGrad, 256>(p, 2, dy, h, d_out, true)))
        return cudaErrorNotSupported;
    // cycles of a tile: its stages, or what its drain takes
    const int64_t deep = 2 * PARTS * p.q[0].depth * kStageCycles;
    const int64_t depth = PARTS * (q.d_in ? p.q[1].depth : p.q[2].depth);
    const int64_t flat = depth * kStageCycles > kDrainCycles ? depth * kStageCycles : kDrainCycles;
    p.rounds = (uint32_t)((deep + flat / 2) / flat);
    return launch_product<T, kGrad, 0, 256, 1>(p, s);
}

template <class T, int ACT>
cudaError_t forward(const FfnParams& q, cudaStream_t s)
{
    // few:: has two parts up to kPartsTokens
    if (q.tokens <= (q.parts == 2 ? kPartsTokens : kFewTokens)) return few::forward<T, ACT>(q, s);
    return q.parts == 2 ? forward<T, ACT, 2>(q, s) : forward<T, ACT, 1>(q, s);
}

template <class T, int ACT>
cudaError_t backward(const FfnBackParams& q, cudaStream_t s)
{
    return q.parts == 2 ? backward<T, ACT, 2>(q, s) : backward<T, ACT, 1>(q, s);
}

template <class T>
cudaError_t forward(const FfnParams& q, cudaStream_t s)
{
    return q.act == PTOC_ACT_SILU ? forward<T, PTOC_ACT_SILU>(q, s) : forward<T, PTOC_ACT_GELU>(q, s);
}

template <class T>
cudaError_t backward(const FfnBackParams& q, cudaStream_t s)
{
    return q.act == PTOC_ACT_SILU ? backward<T, PTOC_ACT_SILU>(q, s) : backward<T, PTOC_ACT_GELU>(q, s);
}

}  // namespace

}  // namespace ptoc
