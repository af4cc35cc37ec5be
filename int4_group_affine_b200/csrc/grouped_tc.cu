// grouped_tc.cu - products grouped by expert with ragged sizes, and their gradients, on the tcgen05
// tensor cores (sm_100a): operands by TMA, accumulators in tensor memory.
//
// One persistent kernel for the three directions.  A tile of the output is 256 matrix rows (the
// tensor memory's lanes of two blocks) by up to 256 columns, over the sum in steps of 64:
//
//   forward  lanes = outputs n of W[g], columns = rows m of the group, sum over k
//   dx       lanes = inputs k of W[g],  columns = rows m of the group, sum over n
//   dw       lanes = outputs n,         columns = inputs k,            sum over the group's rows m
//
// With the matrix on the lanes, the ragged side is the one whose width the instruction can choose: a
// group of c rows takes ceil(c / 256) tiles of equal width, rounded up to 32, so a group of 17 rows
// multiplies 32 columns and not 128.  An operand whose summed index is contiguous in memory (W and x
// in the forward, dy in dx) is stored K-major, the others (W in dx; dy and x in dw) MN-major: the
// 128-byte-swizzled boxes that TMA writes are the tensor core's own layout for either, so nothing is
// transposed by hand.
//
// Weight gradients of few tiles and many rows: a cluster of up to eight blocks shares a tile's rows,
// each leaves its sums in shared memory where the operands were, and each adds up its part of the
// columns from all of them, in order.
//
// Forward and dx share a tile between a cluster's two blocks (cta_group::2): each loads its 128 lanes
// and half of the columns, a third fewer bytes than two tiles of 128 x 256 take (7 % on 16 groups of
// about 960 rows).  Matrices of 128 outputs or fewer, and dw, run on single blocks: in dw every tile
// ends with a clean-up (below) that a pair has to hand across (178 us against 139).
//
// Rows of other groups.  The row boxes run past a group's end.  In forward and dx those rows only
// fill columns that are not stored.  In dw they would enter the sum, so the MMA warp clears them in
// both operands (a NaN times zero is a NaN) up to the next 16, and multiplies no further.
//
// Warps: 0 loads (TMA, one box an operand and step, into a ring of six 32 KB stages, four of 48 KB on
// single blocks; calls of few rows into five of two steps each, below), 1 multiplies
// (tcgen05.mma), 2..9 write results, two per quarter of the lanes; the accumulator is double buffered,
// so a tile is written while the next one multiplies.  Forward and dx: neighbouring lanes exchange
// halves, and a warp stores two rows' 64-byte pieces at a time.  dw: 32 x 128-byte boxes through
// shared memory and TMA stores, which clip at the matrix's edges.  Every wait is bounded.
//
// What bounds it.  The loop: a stage's products take 512 cycles at full width, and a warp issues an
// instruction in 5 to 20 cycles, so the two pipeline warps run uniform, short loops with one elected
// lane issuing, and a step's operands are one request each (with the columns in boxes of falling powers
// of two, up to three a step, the row gradient below took 76 us).  Whole calls: many small groups run
// at the speed of the memory (16,380 rows on 256 experts of 1024 x 2048: 177 us, 6.6 TB/s), large ones
// at the tensor cores' and the power limit (16384 rows on 16 experts, row gradient: 68 us), the fp32
// weight gradient at its stores and loads, which overlap in part (64 x 1024 x 2048: 124 to 147 us, 97 for the
// stores alone, 93 without them).
//
// Long sums: the tensor core's accumulation rounds toward zero, an error that grows with the sum's
// length (measured 4.7e-7 of the result at 512 terms, 9.1e-6 at 8192; 4.5e-4 at 65536 of one sign, as
// much as a rounding to fp16).  Sums of fp32 weight gradients longer than 512 rows leave the tensor
// core in parts and are added by the L2's fp32 additions, one part after the other (a fixed order), or
// by the result warps where an earlier gradient is to meet the complete sum; those for 16-bit results
// leave it every 8192 terms and are added up in fp32 by the result warps.
#include <cuda_fp16.h>
#include <cudaTypedefs.h>

#include <algorithm>

#include "grouped.cuh"
#include "tc.cuh"

namespace moeq {
namespace {

constexpr int kLanes = 128;              // matrix rows of a block's part of a tile
constexpr int kCols = 256;               // and at most this many columns
constexpr int kStep = 64;                // terms per 128-byte box
constexpr int kABytes = kLanes * 128;    // 64 16-bit terms of every lane
constexpr int kBox = 64 * 128;           // an MN-major box: 64 terms of 64 outputs
constexpr int kEpi = 8;                  // result warps
constexpr int kThreads = (2 + kEpi) * 32;
constexpr int kOutBytes = 32 * 128;      // dw: a warp's staging box
constexpr int kPart = 512;               // fp32 dw: terms per part
constexpr int kPart16 = 8192;            // the others (the error of so many is a small part of their rounding)

// Calls of so few rows take stages of two steps: the ring's upkeep (300 cycles a stage) is what a block's tile of few
// columns takes, not its products (30 cycles for 16 terms).  34 rows on 256 experts of 1024 x 2048: 24.5 us, with stages
// of one step 26.3; 8 rows 11.9 and 13.8 (both less 0.9 by now); 60 rows on 8 of 4096 x 4096 46 and 49 (of all that was timed one call lost:
// the row gradient of 64 rows on 64 experts of 512 x 4096, 32.5 and 30.0).
constexpr int kNarrowRows = 64;

// Shared memory by direction and by the blocks that share a tile (kCta = 2: a cluster's pair, each loading its 128
// rows and half of the columns).
template <int kDir, int kCta, int kNarrow>
struct Ring {
    static constexpr int outs = kDir == kGmmDw ? 1 : 0;  // a result warp's staging boxes
    static constexpr int steps = kNarrow ? 2 : 1;        // of a stage
    static constexpr int stages = kNarrow ? 5 : kCta == 2 ? 6 : 4;
    static constexpr int col_bytes = (kNarrow ? kNarrowRows : kCols) / kCta * 128;  // the columns' operand, of a step
    static constexpr int bytes = steps * (kABytes + col_bytes);
    static constexpr size_t smem = 1024 + stages * bytes + outs * kEpi * kOutBytes;
    static_assert(col_bytes % 1024 == 0 && smem + (kDir == kGmmDw ? 1024 : 10 * 1024) <= 227 * 1024, "shared memory");
};

constexpr int kBoxes = 8;

struct TcGmm {
    CUtensorMap tma;     // the lanes' operand
    CUtensorMap tmb[kBoxes];  // the columns' operand: forward, dx in boxes of 1 .. 8 times 16 rows (single blocks 32); dw [0]
    CUtensorMap tmo;     // dw: the output, in boxes of 32 rows x 128 bytes
    int table;           // forward, dx: the groups fit the block's table
    // forward, dx: the lane blocks of the output, and those of all parts of the sum; dw: the column blocks of a group and
    // its tiles; and their reciprocals
    int real, across;
    float inv_real, inv;
    int wide_a, wide_b;  // an MN-major operand whose whole tile is one box (see encode_mn)
    GmmArgs a;
};

// A tile of work as every warp role sees it.
struct Tile {
    int g;         // group (-1: no more)
    int lane0;     // first output row of the tile
    int col0;      // first column: row of x / dy (forward, dx), input k (dw)
    int cols;      // columns that count
    int width;     // columns multiplied: cols rounded up
    int terms;     // the sum runs to this term
    int first;     // from this one on (0 but where the sum is split)
    int part;      // and is this part of it
    int row0;      // dw: first row of the group
};

// The groups' tiles, worked out once a block for up to kTable groups whose offsets are in order (others walk the
// offsets as they go): finding a tile's group takes two looks instead of one for every 32 groups before it.
constexpr int kTable = 1024;
struct Table {
    int off[kTable + 1];
    int upto[kTable];         // tiles up to and with a group, counted from its window of 32 groups
    int before[kTable / 32];  // tiles before a window
    int total;
};

// Fills the table (all threads of the block); false where the offsets are not in order (the table is of no use then).
template <int kThreads>
__device__ __forceinline__ bool fill_table(Table& tb, const GmmArgs& a, int across, int tid) {
    const int warp = tid / 32, lane = tid % 32, windows = (a.G + 31) / 32;
    for (int i = tid; i <= a.G; i += kThreads) tb.off[i] = ld_after(a.off + i);
    __syncthreads();
    bool good = true;
    for (int i = tid; i <= a.G; i += kThreads) good = good && tb.off[i] >= (i > 0 ? tb.off[i - 1] : 0) && tb.off[i] <= a.M;
    if (!good && blockIdx.x == 0) raise_status(a.status, MOE_ERR_DEVICE_INDEX);
    for (int w = warp; w < windows; w += kThreads / 32) {
        const int g = 32 * w + lane;
        int t = g < a.G ? (tb.off[g + 1] - tb.off[g] + kCols - 1) / kCols * across : 0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, t, o);
            if (lane >= o) t += v;
        }
        tb.upto[g] = t;
        if (lane == 31) tb.before[w] = t;
    }
    good = __syncthreads_and(good);
    if (warp == 0) {
        int t = lane < windows ? tb.before[lane] : 0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, t, o);
            if (lane >= o) t += v;
        }
        if (lane == windows - 1) tb.total = t;
        t = __shfl_up_sync(0xffffffffu, t, 1);
        if (lane < windows) tb.before[lane] = lane ? t : 0;
    }
    __syncthreads();
    return good;
}

// The group that owns `tile` (a warp; there is one), its rows and the tile's index within it.
__device__ __forceinline__ int find_in(const Table& tb, int G, int64_t tile, int lane, GmmRows* rows, int* within) {
    const int windows = (G + 31) / 32;
    const uint32_t m = __ballot_sync(0xffffffffu, lane < windows && tile >= tb.before[min(lane, windows - 1)]);
    const int w = 31 - __clz(m), rest = (int)(tile - tb.before[w]);  // (window 0 begins with tile 0)
    const int upto = tb.upto[32 * w + lane];
    const uint32_t in = __ballot_sync(0xffffffffu, rest < upto);
    const int l = __ffs(in) - 1, g = 32 * w + l;
    *rows = GmmRows{tb.off[g], tb.off[g + 1]};
    *within = rest - (l > 0 ? __shfl_sync(0xffffffffu, upto, l - 1) : 0);
    return g;
}

// n / d and n % d for small n (a quotient below 2^22), without the integer division's hundred instructions.
struct Quot {
    int q, r;
};
__device__ __forceinline__ Quot quot(int n, int d, float inv) {
    int q = (int)((float)n * inv), r = n - q * d;
    while (r < 0) --q, r += d;
    while (r >= d) ++q, r -= d;
    return Quot{q, r};
}

// The tiles of a block (or pair), one after the other.  Every warp role walks them for itself, and a tile of a small
// group is over in 2,000 cycles: tile indices advance by additions, and a group is looked up once.
template <int kDir, int kCta>
struct Schedule {
    static constexpr int kTileLanes = kLanes * kCta;
    static constexpr int kUp = 16 * kCta;  // what the instruction's width is a multiple of
    GmmWalk walk;
    GmmRows rows;                          // (dw: as read, ahead of the tile)
    const Table* table;                    // forward, dx: or NULL
    bool good;
    int g = -1, across, left;              // left: tiles (forward, dx: of this group) from this one on
    int within, step, step_g;              // dw: tile within the group, and the stride in groups and tiles
    int share, shares;                     // dw: of a tile's rows this block sums up share / shares
    int parts, width;                      // forward, dx: tiles along the group's rows, and their width
    int64_t tile;
    int total;                             // with a table: all tiles
    int real;                              // forward, dx: lane blocks of a part of the sum
    float inv, inv_real;

    __device__ __forceinline__ void start(const TcGmm& p, int first, int stride, int lane, bool good_, const Table* table_) {
        good = good_;
        table = table_;
        real = p.real, across = p.across;
        inv_real = p.inv_real, inv = p.inv;
        if (kDir == kGmmDw) {
            left = real;  // tiles of a group
            const Quot q = quot(first, left, inv_real), s = quot(stride, left, inv_real);
            g = q.q, within = q.r;
            step_g = s.q, step = s.r;
            share = 0, shares = 1;
            fetch(p.a, lane);
        } else {
            total = table ? table->total : 0;
            tile = first;
            step = stride;
            left = 0;
        }
    }

    // dw: the rows of group g, on their way while the tile before them is worked on.
    __device__ __forceinline__ void fetch(const GmmArgs& a, int lane) {
        if (g >= a.G) return;
        if (!good) rows = gmm_rows_of(a, g, lane);
        else rows = a.off ? GmmRows{ld_after(a.off + g), ld_after(a.off + g + 1)} : GmmRows{0, a.M};
    }

    // The next tile; g = -1 when there is none.
    __device__ __forceinline__ Tile next(const GmmArgs& a, int lane) {
        Tile t;
        if (kDir == kGmmDw) {
            t.g = g < a.G ? g : -1;
            if (t.g < 0) return t;
            const Quot p = quot(within, across, inv);
            t.lane0 = p.q * kTileLanes;
            t.col0 = p.r * kCols;
            t.cols = min(kCols, a.K - t.col0);
            t.width = (t.cols + kUp - 1) & ~(kUp - 1);
            t.terms = rows.end - rows.begin;
            t.first = t.part = 0;
            t.row0 = rows.begin;
            if (shares > 1) {
                const int per = ((t.terms + kStep - 1) / kStep + shares - 1) / shares * kStep;
                t.row0 += min(share * per, t.terms);
                t.terms = min(max(t.terms - share * per, 0), per);
            }
            within += step;
            int ng = g + step_g;
            if (within >= left) within -= left, ++ng;
            if (ng != g) {
                g = ng;
                fetch(a, lane);
            }
        } else {
            if (left <= 0) {  // another group
                if (table) {
                    t.g = -1;
                    if (tile >= total) return t;
                    g = find_in(*table, a.G, tile, lane, &rows, &within);
                } else {
                    int64_t w = 0;
                    g = walk.find(a, lane, tile, kCols, across, &rows, &w);
                    within = (int)w;
                }
                t.g = g;
                if (g < 0) return t;
                const int count = rows.end - rows.begin;
                parts = (count + kCols - 1) / kCols;
                width = parts == 1 ? count : (count + parts - 1) / parts;
                width = (width + kUp - 1) & ~(kUp - 1);
                left = parts * across - within;
            }
            t.g = g;
            const Quot p = quot(within, across, inv);
            const Quot l = a.splits > 1 ? quot(p.r, real, inv_real) : Quot{0, p.r};
            t.part = l.q;
            t.lane0 = l.r * kTileLanes;
            t.col0 = rows.begin + p.q * width;
            t.cols = min(width, rows.end - t.col0);
            t.terms = kDir == kGmmFwd ? a.K : a.N;
            t.first = 0;
            if (a.splits > 1) {
                t.first = t.part * a.per;
                t.terms = min(t.terms, t.first + a.per);
            }
            t.width = (t.cols + kUp - 1) & ~(kUp - 1);
            within += step;
            left -= step;
            tile += step;
        }
        return t;
    }
};

// The pipeline's two warps run their loops together and one elected lane issues (`one`): the loops' values stay
// uniform, which the tensor core's and TMA's instructions take without a detour.
__device__ __forceinline__ uint32_t elect_one() {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
    return r;
}

// TMA loads into this block's shared memory; a pair's loads may signal a barrier of either block (`bar`: a
// shared::cluster address).
#define MOEQ_TMA_LOAD(dims, coords, ...)                                                                            \
    if (kCta == 2)                                                                                                  \
        asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %3, 0;\n\t@q cp.async.bulk.tensor." dims               \
                     ".shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 [%0], [%1, " coords    \
                     "], [%2];\n\t}" ::"r"(dst),                                                                    \
                     "l"(map), "r"(bar), "r"(one), __VA_ARGS__                                                      \
                     : "memory");                                                                                   \
    else                                                                                                            \
        asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %3, 0;\n\t@q cp.async.bulk.tensor." dims               \
                     ".shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, " coords                 \
                     "], [%2];\n\t}" ::"r"(dst),                                                                    \
                     "l"(map), "r"(bar), "r"(one), __VA_ARGS__                                                      \
                     : "memory")
template <int kCta>
__device__ __forceinline__ void load_2d(uint32_t one, uint32_t dst, const void* map, int x, int y, uint32_t bar) {
    MOEQ_TMA_LOAD("2d", "{%4, %5}", "r"(x), "r"(y));
}
template <int kCta>
__device__ __forceinline__ void load_3d(uint32_t one, uint32_t dst, const void* map, int x, int y, int z, uint32_t bar) {
    MOEQ_TMA_LOAD("3d", "{%4, %5, %6}", "r"(x), "r"(y), "r"(z));
}
template <int kCta>
__device__ __forceinline__ void load_4d(uint32_t one, uint32_t dst, const void* map, int x, int y, int z, int w,
                                        uint32_t bar) {
    MOEQ_TMA_LOAD("4d", "{%4, %5, %6, %7}", "r"(x), "r"(y), "r"(z), "r"(w));
}
#undef MOEQ_TMA_LOAD
__device__ __forceinline__ void expect_tx(uint32_t one, uint32_t bar, uint32_t bytes) {
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %2, 0;\n\t"
        "@q mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n\t}" ::"r"(bar),
        "r"(bytes), "r"(one)
        : "memory");
}

// ------------------------------------------------------------------ pairs of blocks
__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %cluster_ctarank;" : "=r"(r));
    return r;
}
// The address, in the cluster's shared memory, of rank 0's copy of a variable.
__device__ __forceinline__ uint32_t in_rank0(uint32_t addr) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(0));
    return r;
}
// (relaxed: what the tensor memory was read for is in registers by now, and a release would wait for the stores of
// results, which nobody in the cluster reads)
__device__ __forceinline__ void arrive_cluster(uint32_t bar) {
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_arrive_relaxed() { asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory"); }
// A float of the cluster's block `rank`, at this block's shared memory address `addr`.
__device__ __forceinline__ float ld_of(uint32_t addr, int rank) {
    float v;
    asm volatile("{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %1, %2;\n\tld.shared::cluster.f32 %0, [a];\n\t}"
                 : "=f"(v)
                 : "r"(addr), "r"(rank)
                 : "memory");
    return v;
}
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
template <int kCta>
__device__ __forceinline__ void tmem_alloc(uint32_t* dst, uint32_t cols) {  // a warp of every block of the tile
    if (kCta == 1) {
        tc::tmem_alloc(dst, cols);
        tc::tmem_relinquish();
    } else {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(tc::smem_u32(dst)), "r"(cols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
}
template <int kCta>
__device__ __forceinline__ void tmem_free(uint32_t t, uint32_t cols) {
    if (kCta == 1) tc::tmem_dealloc(t, cols);
    else asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(t), "r"(cols) : "memory");
}
// D (+)= A B^T.
template <int kCta>
__device__ __forceinline__ void mma(uint32_t one, uint32_t d, uint64_t ad, uint64_t bd, uint32_t idesc, uint32_t add) {
    if (kCta == 1)
        asm volatile(
            "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
            "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
            "l"(ad), "l"(bd), "r"(idesc), "r"(add), "r"(one)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
            "@q tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
            "l"(ad), "l"(bd), "r"(idesc), "r"(add), "r"(one)
            : "memory");
}
// Arrive on `bar` (of both blocks of a pair) once this thread's MMAs so far are done.
template <int kCta>
__device__ __forceinline__ void commit(uint32_t one, uint32_t bar) {
    if (kCta == 1)
        asm volatile(
            "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
            "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar),
            "r"(one)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
            "@q tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], "
            "%2;\n\t}" ::"r"(bar),
            "r"(one), "h"((uint16_t)3)
            : "memory");
}
// The same on a barrier of this block alone.
template <int kCta>
__device__ __forceinline__ void commit_here(uint32_t bar) {
    if (kCta == 1)
        asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
    else
        asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}

__device__ __forceinline__ void tma_store_3d(uint32_t one, const void* map, uint32_t src, int x, int y, int z) {
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %5, 0;\n\t"
        "@q cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4}], [%1];\n\t}" ::"l"(map),
        "r"(src), "r"(x), "r"(y), "r"(z), "r"(one)
        : "memory");
}
__device__ __forceinline__ void tma_add_3d(uint32_t one, const void* map, uint32_t src, int x, int y, int z) {
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %5, 0;\n\t"
        "@q cp.reduce.async.bulk.tensor.3d.global.shared::cta.add.tile.bulk_group [%0, {%2, %3, %4}], [%1];\n\t}" ::"l"(
            map),
        "r"(src), "r"(x), "r"(y), "r"(z), "r"(one)
        : "memory");
}
// (a whole warp's: the lanes that issue no copy have nothing to wait for)
__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
__device__ __forceinline__ void bulk_wait_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
__device__ __forceinline__ void bulk_wait() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

// 32 lanes x 32 consecutive 32-bit columns.
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr)
        : "memory");
}

// Descriptor of an MN-major operand in 128-byte-swizzled boxes of 64 outputs x 64 terms (a term's 64 outputs are
// one 128-byte row): 8 terms are 1024 bytes apart, the next 64 outputs one box further.
__device__ __forceinline__ uint64_t sdesc_mn_sw128(uint32_t saddr) {
    uint64_t d = 0;
    d |= (uint64_t)((saddr >> 4) & 0x3FFFu);
    d |= (uint64_t)(kBox >> 4) << 16;    // leading byte offset: 64 outputs
    d |= (uint64_t)(1024u >> 4) << 32;   // stride byte offset: 8 terms
    d |= (uint64_t)1u << 46;
    d |= (uint64_t)2u << 61;
    return d;
}

template <int kDir, int kCta>
__device__ __forceinline__ uint32_t idesc_of(int f16, int width) {
    const uint32_t t = f16 ? 0u : 1u;
    return (1u << 4) | (t << 7) | (t << 10) | (kDir != kGmmFwd ? 1u << 15 : 0u) | (kDir == kGmmDw ? 1u << 16 : 0u) |
           ((uint32_t)(width >> 3) << 17) | ((uint32_t)(kLanes * kCta >> 4) << 24);
}

template <int kF16>
__device__ __forceinline__ uint16_t to16(float v) {
    return kF16 ? __half_as_ushort(__float2half_rn(v)) : f2bf16(v);
}
template <int kF16>
__device__ __forceinline__ float from16(uint16_t v) {
    return kF16 ? __half2float(__ushort_as_half(v)) : bf16f(v);
}
template <int kF16>
__device__ __forceinline__ uint32_t pack16(uint32_t lo, uint32_t hi) {  // (fp32 bit patterns)
    const float2 v = make_float2(__uint_as_float(lo), __uint_as_float(hi));
    if (kF16) {
        const __half2 h = __float22half2_rn(v);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
    const __nv_bfloat162 b = __float22bfloat162_rn(v);
    return *reinterpret_cast<const uint32_t*>(&b);
}

// As tc::mbar_wait_ok, for after a first try: out of the loops' code, with the device's clock (slow to read) and the
// flag looked at once in 256 tries.  (A lone warp issues an instruction in 5 to 20 cycles and a stage's products take
// 512 at most: with the waits in line and the values in one thread's registers the loops took 1,070.)
__device__ __noinline__ bool wait_more(uint64_t* bar, uint32_t parity, int32_t* status, volatile int* ok, uint64_t limit) {
    uint64_t t0 = 0;
    for (;;) {
        for (int i = 0; i < 256; ++i)
            if (tc::mbar_try_wait(bar, parity)) return true;
        const uint64_t t = tc::globaltimer_ns();
        if (*ok == 0) return false;
        if (t0 == 0) t0 = t;
        if (t - t0 > limit) break;
    }
    raise_status(status, MOE_ERR_TIMEOUT);
    *ok = 0;
    return false;
}
// A whole warp's wait: the same answer in every lane, so that a wait that gives up never splits the warp.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, const GmmArgs& a, volatile int* ok) {
    if (__all_sync(0xffffffffu, tc::mbar_try_wait(bar, parity))) return true;
    return __all_sync(0xffffffffu, wait_more(bar, parity, a.status, ok, a.wait_ns));
}

// The bound of a block's last waits: what is under way ends by itself, also where the waits before were cut short.
__device__ __forceinline__ uint64_t drain_ns(const GmmArgs& a) { return a.wait_ns > 1000000000ull ? a.wait_ns : 1000000000ull; }

// A millisecond, for what is under way and cannot be waited for after the blocks have given up.
__device__ __forceinline__ void let_pass() {
    for (const uint64_t t0 = tc::globaltimer_ns(); tc::globaltimer_ns() - t0 < 1000000;) {
    }
}

// A place in the ring of stages, and the parity its barriers complete with next.
template <int kStages>
struct Place {
    uint32_t st = 0, phase = 0;
    __device__ __forceinline__ void next() {
        if (++st == kStages) st = 0, phase ^= 1;
    }
};

// kSplit: the a.splits blocks of a cluster share the rows of a tile (weight gradients; one tile a cluster).
template <int kDir, int kF16, int kCta, int kNarrow, int kSplit>
__global__ void __launch_bounds__(kThreads, 1) gmm_tc_kernel(const __grid_constant__ TcGmm p) {
    using R = Ring<kDir, kCta, kNarrow>;
    constexpr int kStages = R::stages, kStageBytes = R::bytes, kTerms = kStep * R::steps;  // terms of a stage
    static_assert(kDir != kGmmDw || kCta == 1, "dw clears operands behind the group's last row: a block's own");
    extern __shared__ unsigned char raw[];
    unsigned char* sm = raw + ((1024u - (tc::smem_u32(raw) & 1023u)) & 1023u);
    unsigned char* s_out = sm + kStages * kStageBytes;
    __shared__ uint64_t bar_full[kStages], bar_empty[kStages];  // a stage landed / was multiplied
    __shared__ uint64_t bar_acc[2], bar_free[2];                // an accumulator is complete / was read
    __shared__ uint64_t bar_drain;
    __shared__ uint32_t s_tmem;
    __shared__ volatile int s_ok;
    __shared__ Table s_table;
    const GmmArgs& a = p.a;
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    const int rank = kCta == 2 ? (int)cluster_rank() : 0;

    if (warp == 1) tmem_alloc<kCta>(&s_tmem, 512);
    if (tid == 0) {
        for (int i = 0; i < kStages; ++i) {
            tc::mbar_init(&bar_full[i], 1);
            tc::mbar_init(&bar_empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            tc::mbar_init(&bar_acc[i], 1);
            tc::mbar_init(&bar_free[i], kEpi * kCta);
        }
        tc::mbar_init(&bar_drain, 1);
        tc::mbar_init_fence();
        s_ok = 1;
        tc::tma_prefetch_desc(&p.tma);
        tc::tma_prefetch_desc(&p.tmb[0]);
        if (kDir == kGmmDw) tc::tma_prefetch_desc(&p.tmo);
    }
    __syncwarp();
    if (kCta == 2) cluster_arrive();
    // The next kernel may set itself up beside this one, whose blocks leave room for no second of their kind (8 rows on 64
    // experts of 512 x 512, again and again: 5.8 us, without 6.2; kernels that share an SM crowd on its first free ones).
    grid_release();
    grid_wait();
    // whether the offsets are in order, so that a group's rows need no look at the groups before it
    bool good = true;
    tc::tc_fence_before();
    if (kDir != kGmmDw && p.table) {
        good = fill_table<kThreads>(s_table, a, p.across, tid);
    } else {
        if (kDir == kGmmDw || blockIdx.x == 0) good = gmm_check_offsets(a, tid, kThreads);
        good = __syncthreads_and(good);
    }
    if (kCta == 2) cluster_wait();
    tc::tc_fence_after();
    const uint32_t tmem = s_tmem;
    const uint32_t sbase = tc::smem_u32(sm);
    Schedule<kDir, kCta> sched;
    const int team = kSplit ? a.splits : kCta;  // blocks of a tile
    sched.start(p, blockIdx.x / team, gridDim.x / team, lane, good, kDir != kGmmDw && p.table && good ? &s_table : nullptr);
    if (kSplit) sched.share = blockIdx.x % team, sched.shares = team;
    const int part = kDir == kGmmDw && a.out_f32 ? kPart : kPart16;  // long sums in parts

    if (warp == 0) {
        // ------------------------------------------------------------ loads
        Place<kStages> at;
        uint32_t n = 0;  // stages issued
        const uint32_t own0 = tc::smem_u32(bar_full), full0 = kCta == 2 ? in_rank0(own0) : own0;
        const uint32_t one = elect_one();
        bool ok = true;
        while (ok) {
            const Tile t = sched.next(a, lane);
            if (t.g < 0) break;
            const int lanes = t.lane0 + kLanes * rank, half = t.width / kCta, col = t.col0 + half * rank;
            const int bk = (half + 63) / 64;  // dw: boxes of 64 columns
            constexpr int kUnit = kCols / kCta / kBoxes;
            const int units = (half + kUnit - 1) / kUnit;  // forward, dx: one box of so many rows
            const CUtensorMap* const mapb = &p.tmb[kDir == kGmmDw ? 0 : units - 1];
            const uint32_t bytes = R::steps * (kABytes + (kDir == kGmmDw ? (p.wide_b ? kCols / 64 : bk) * kBox : units * (kUnit * 128)));
            for (int k0 = t.first; k0 < t.terms; k0 += kTerms, at.next(), ++n) {
                ok = warp_wait(&bar_empty[at.st], at.phase ^ 1, a, &s_ok);  // (free from the start)
                if (!ok) break;
                const uint32_t full = full0 + 8 * at.st;
                if (rank == 0) expect_tx(one, own0 + 8 * at.st, kCta * bytes);
#pragma unroll
                for (int i = 0; i < R::steps; ++i) {
                    const int k = k0 + i * kStep;  // (a second step behind the last term reads as zeros, or is not multiplied)
                    const uint32_t sa = sbase + at.st * kStageBytes + i * kABytes;
                    const uint32_t sb = sbase + at.st * kStageBytes + R::steps * kABytes + i * R::col_bytes;
                    if (kDir == kGmmFwd) {
                        load_3d<kCta>(one, sa, &p.tma, k, lanes, t.g, full);
                    } else if (kDir == kGmmDx) {
                        if (p.wide_a) {
                            load_4d<kCta>(one, sa, &p.tma, 0, k, lanes / 64, t.g, full);
                        } else {
                            load_3d<kCta>(one, sa, &p.tma, lanes, k, t.g, full);
                            load_3d<kCta>(one, sa + kBox, &p.tma, lanes + 64, k, t.g, full);
                        }
                    } else if (p.wide_a) {
                        load_3d<kCta>(one, sa, &p.tma, 0, t.row0 + k, lanes / 64, full);
                    } else {
                        load_2d<kCta>(one, sa, &p.tma, lanes, t.row0 + k, full);
                        load_2d<kCta>(one, sa + kBox, &p.tma, lanes + 64, t.row0 + k, full);
                    }
                    if (kDir == kGmmDw) {
                        if (p.wide_b) {
                            load_3d<kCta>(one, sb, &p.tmb[0], 0, t.row0 + k, col / 64, full);
                        } else {
                            for (int i = 0; i < bk; ++i)
                                load_2d<kCta>(one, sb + i * kBox, &p.tmb[0], col + 64 * i, t.row0 + k, full);
                        }
                    } else {
                        load_2d<kCta>(one, sb, mapb, k, col, full);
                    }
                }
            }
        }
        // No block ends with copies on their way into it, or the tensor core's reports that a stage was multiplied, which
        // a pair's first block sends to both.  (A pair's copies report to its first block, and a stage that was multiplied
        // had landed; should the two have parted in giving up, what is left cannot be told and gets time to pass.)
        if (one) {
            const uint32_t last = n > kStages ? n - kStages : 0;
            if (rank == 0)
                for (uint32_t i = last; i < n; ++i)
                    tc::mbar_wait(&bar_full[i % kStages], (i / kStages) & 1, a.status, drain_ns(a));
            bool all = ok;
            for (uint32_t i = last; all && i < n; ++i)
                all = tc::mbar_wait_ok(&bar_empty[i % kStages], (i / kStages) & 1, a.status, &s_ok, drain_ns(a));
            if (!all) let_pass();
        }
    } else if (warp == 1 && rank == 0) {
        // ------------------------------------------------------------ products
        // descriptors of stage 0; a stage, and 16 terms, are so many 16-byte units further
        constexpr uint32_t kAdvA = kDir == kGmmFwd ? 32 >> 4 : 2048 >> 4, kAdvB = kDir == kGmmDw ? 2048 >> 4 : 32 >> 4;
        const uint64_t ad0 = kDir == kGmmFwd ? tc::sdesc_k_sw128(sbase) : sdesc_mn_sw128(sbase);
        const uint64_t bd0 = kDir == kGmmDw ? sdesc_mn_sw128(sbase + kABytes) : tc::sdesc_k_sw128(sbase + R::steps * kABytes);
        const uint32_t empty0 = tc::smem_u32(bar_empty), acc0 = tc::smem_u32(bar_acc);
        const uint32_t one = elect_one();
        Place<kStages> at;
        uint32_t acc = 0;
        bool ok = true;
        while (ok) {
            const Tile t = sched.next(a, lane);
            if (t.g < 0) break;
            const uint32_t idesc = idesc_of<kDir, kCta>(kF16, t.width);
            for (int p0 = t.first; ok && p0 < t.terms; ++acc) {
                const int p1 = min(t.terms, p0 + part);
                const uint32_t d = tmem + (acc & 1) * kCols;
                ok = warp_wait(&bar_free[acc & 1], (acc / 2 & 1) ^ 1, a, &s_ok);
                if (!ok) break;
                tc::tc_fence_after();
                for (int k = p0; k < p1; k += kTerms, at.next()) {
                    ok = warp_wait(&bar_full[at.st], at.phase, a, &s_ok);
                    if (!ok) break;
                    const int left = t.terms - k;
                    if (kDir == kGmmDw && left < kStep && left % 16) {  // the rows behind the group's last
                        unsigned char* base = sm + at.st * kStageBytes + lane * 16;
                        const int end = left + 15 & ~15;
                        for (int r = left; r < end; r += 4)  // four 128-byte rows of every box at a time
                            if (r + lane / 8 < end) {
#pragma unroll
                                for (int b = 0; b < kStageBytes / kBox; ++b)
                                    *reinterpret_cast<uint4*>(base + b * kBox + r * 128) = make_uint4(0, 0, 0, 0);
                            }
                        tc::fence_async_smem();
                        __syncwarp();
                    }
                    tc::tc_fence_after();
                    const uint64_t ad = ad0 + at.st * (kStageBytes >> 4), bd = bd0 + at.st * (kStageBytes >> 4);
                    auto terms16 = [&](int s) {
                        mma<kCta>(one, d, ad + s % 4 * kAdvA + s / 4 * (kABytes >> 4),
                                  bd + s % 4 * kAdvB + s / 4 * (R::col_bytes >> 4), idesc, s > 0 || k > p0);
                    };
                    if (left >= kTerms) {
#pragma unroll
                        for (int s = 0; s < kTerms / 16; ++s) terms16(s);
                    } else {
                        for (int s = 0; 16 * s < left; ++s) terms16(s);
                    }
                    commit<kCta>(one, empty0 + 8 * at.st);
                }
                if (ok) commit<kCta>(one, acc0 + 8 * (acc & 1));
                p0 = p1;
            }
        }
        // and none with products under way, or the second block's reports that it has read an accumulator
        if (kCta == 2) {
            bool all = ok;
            for (uint32_t i = acc > 2 ? acc - 2 : 0; all && i < acc; ++i) all = warp_wait(&bar_free[i & 1], i / 2 & 1, a, &s_ok);
            if (one && !all) let_pass();
        }
        if (one) {
            commit_here<kCta>(tc::smem_u32(&bar_drain));
            tc::mbar_wait(&bar_drain, 0, a.status, drain_ns(a));
        }
    } else if (warp > 1) {
        // ------------------------------------------------------------ results
        const int q = warp % 4, half = (warp - 2) / 4;  // lanes [32 q, 32 q + 32), every other piece of columns
        uint32_t acc = 0;
        bool ok = true;
        auto release = [&](uint64_t* bar) {  // an accumulator may be overwritten, as far as this warp goes
            if (kCta == 2) arrive_cluster(in_rank0(tc::smem_u32(bar)));
            else tc::mbar_arrive(bar);
        };
        unsigned char* sg = s_out + (warp - 2) * kOutBytes;  // dw: the staging box
        const uint32_t so = tc::smem_u32(sg), one = elect_one();
        const int J = kDir == kGmmFwd ? a.N : a.K;
        const bool pairs = J % 2 == 0 && (reinterpret_cast<uintptr_t>(a.out) & 3) == 0;
        const uint32_t own = tmem + ((uint32_t)(32 * q) << 16);  // this warp's lanes
        // Parts of a long sum before its last are added up here, `band` columns of every other band, those of the pieces
        // that the warp writes (in local memory: few sums are so long).  fp32 weight gradients that nothing is added to
        // leave their parts to the L2's additions (20000 rows, 2048 x 2048: 229 us, added up here 252; 200 groups of 700
        // rows, 64 x 64: 13.1 and 14.0).
        constexpr int kBand = kDir == kGmmDw ? 64 : 32;
        const bool fp32 = kDir == kGmmDw && !kSplit && a.out_f32, in_memory = fp32 && !a.accumulate;
        const int band = fp32 ? 32 : kBand;
        float sum[kCols / 2];
        while (ok) {
            const Tile t = sched.next(a, lane);
            if (t.g < 0) break;
            int p0 = t.first;
            if (!in_memory)
                for (; ok && t.terms - p0 > part; p0 += part, ++acc) {
                    ok = warp_wait(&bar_acc[acc & 1], (acc / 2) & 1, a, &s_ok);
                    if (!ok) break;
                    tc::tc_fence_after();
                    float* to = sum;
                    for (int c0 = band * half; c0 < t.cols; c0 += 2 * band)
                        for (int c = c0; c < c0 + band; c += 32, to += 32) {
                            uint32_t v[32];
                            tmem_ld32(own + (acc & 1) * kCols + c, v);
                            tc::tmem_wait_ld();
                            for (int j = 0; j < 32; ++j) to[j] = __uint_as_float(v[j]) + (p0 > t.first ? to[j] : 0.0f);
                        }
                    tc::tc_fence_before();
                    __syncwarp();
                    if (lane == 0) release(&bar_free[acc & 1]);
                }
            if (!ok) break;
            if (kDir != kGmmDw) {
                ok = warp_wait(&bar_acc[acc & 1], (acc / 2) & 1, a, &s_ok);
                if (!ok) break;
                tc::tc_fence_after();
                const int f = t.lane0 + kLanes * rank + 32 * q + lane;
                const uint32_t d = own + (acc & 1) * kCols;
                uint16_t* out = reinterpret_cast<uint16_t*>(a.out) + (int64_t)t.col0 * J;
                for (int c = 32 * half; c < t.cols; c += 64) {
                    uint32_t v[32];
                    tmem_ld32(d + c, v);
                    tc::tmem_wait_ld();
                    if (p0 > t.first)
                        for (int j = 0; j < 32; ++j) v[j] = __float_as_uint(__uint_as_float(v[j]) + sum[c / 64 * 32 + j]);
                    const int live = f < J ? t.cols - c : 0;
                    if (a.splits > 1) {
                        float* o = a.partial + ((int64_t)t.part * a.M + t.col0 + c) * J + f;
#pragma unroll
                        for (int i = 0; i < 32; ++i) {
                            if (i < live) *o = __uint_as_float(v[i]);
                            o += J;
                        }
                    } else if (pairs) {
                        // neighbouring lanes exchange, so that each stores two outputs of one row: the even lane
                        // of the first of two rows, the odd lane of the second
                        uint16_t* o = out + (int64_t)(c + (lane & 1)) * J + (f & ~1);
                        const uint32_t pick = lane & 1 ? 0x3276u : 0x5410u;
#pragma unroll
                        for (int i = 0; i < 32; i += 2) {
                            const uint32_t mine = pack16<kF16>(v[i], v[i + 1]);
                            const uint32_t two = __byte_perm(mine, __shfl_xor_sync(0xffffffffu, mine, 1), pick);
                            if (i + (lane & 1) < live) *reinterpret_cast<uint32_t*>(o) = two;
                            o += 2 * J;
                        }
                    } else {
                        uint16_t* o = out + (int64_t)c * J + f;
#pragma unroll
                        for (int i = 0; i < 32; ++i) {
                            if (i < live) *o = to16<kF16>(__uint_as_float(v[i]));
                            o += J;
                        }
                    }
                }
                tc::tc_fence_before();
                __syncwarp();
                if (lane == 0) release(&bar_free[acc & 1]);
                ++acc;
                continue;
            }
            // dw: pieces of 128 bytes of every lane's row (32 fp32 or 64 16-bit columns)
            const int n0 = t.lane0 + kLanes * rank + 32 * q, n = n0 + lane;
            const int per = a.out_f32 ? 32 : 64;
            const bool empty = t.terms == 0;
            if (kSplit) {  // this block's sums, to where the operands were: [column][row of the tile]
                if (!empty) {
                    ok = warp_wait(&bar_acc[acc & 1], (acc / 2) & 1, a, &s_ok);
                    if (!ok) break;
                    tc::tc_fence_after();
                }
                for (int c0 = kBand * half; c0 < t.cols; c0 += 2 * kBand)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        float* to = reinterpret_cast<float*>(sm) + (c0 + 32 * h) * kLanes + 32 * q + lane;
                        uint32_t v[32];
                        if (!empty) {
                            tmem_ld32(own + (acc & 1) * kCols + c0 + 32 * h, v);
                            tc::tmem_wait_ld();
                        }
#pragma unroll
                        for (int j = 0; j < 32; ++j) {
                            float f = empty ? 0.0f : __uint_as_float(v[j]);
                            if (p0 > 0) f += sum[c0 / 128 * 64 + 32 * h + j];
                            to[j * kLanes] = f;
                        }
                    }
                break;
            }
            if (empty && a.accumulate) continue;
            while (ok && (p0 < t.terms || empty)) {
                const bool later = in_memory && p0 > 0, add = a.accumulate || later;  // (a part behind the first)
                const uint32_t buf = acc & 1;
                if (!empty) {
                    ok = warp_wait(&bar_acc[buf], (acc / 2) & 1, a, &s_ok);
                    if (!ok) break;
                    tc::tc_fence_after();
                }
                for (int c = per * half; c < t.cols; c += 2 * per) {
                    uint32_t w[32];
                    if (empty) {
#pragma unroll
                        for (int i = 0; i < 32; ++i) w[i] = 0;
                    } else if (a.out_f32) {
                        tmem_ld32(own + buf * kCols + c, w);
                        tc::tmem_wait_ld();
                        if (p0 > 0 && !later)
                            for (int j = 0; j < 32; ++j) w[j] = __float_as_uint(__uint_as_float(w[j]) + sum[c / 64 * 32 + j]);
                    } else {
                        uint32_t vv[2][32];
                        tmem_ld32(own + buf * kCols + c, vv[0]);
                        tmem_ld32(own + buf * kCols + c + 32, vv[1]);
                        tc::tmem_wait_ld();
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            uint32_t(&v)[32] = vv[h];
                            if (p0 > 0)
                                for (int j = 0; j < 32; ++j)
                                    v[j] = __float_as_uint(__uint_as_float(v[j]) + sum[c / 128 * 64 + 32 * h + j]);
                            if (add) {  // the earlier gradient, added in fp32 and rounded once
                                const uint16_t* old = reinterpret_cast<const uint16_t*>(a.out) +
                                                      ((int64_t)t.g * a.N + n) * a.K + t.col0 + c + 32 * h;
#pragma unroll
                                for (int i = 0; i < 4; ++i) {
                                    if (n >= a.N || t.col0 + c + 32 * h + 8 * i >= a.K) continue;
                                    const uint4 u = *reinterpret_cast<const uint4*>(old + 8 * i);
                                    const uint32_t e[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                                    for (int j = 0; j < 4; ++j) {
                                        float* lo = reinterpret_cast<float*>(&v[8 * i + 2 * j]);
                                        lo[0] += from16<kF16>((uint16_t)(e[j] & 0xFFFFu));
                                        lo[1] += from16<kF16>((uint16_t)(e[j] >> 16));
                                    }
                                }
                            }
#pragma unroll
                            for (int i = 0; i < 16; ++i)
                                w[16 * h + i] = pack16<kF16>(v[2 * i], v[2 * i + 1]);
                        }
                    }
                    // the staging box is free, and earlier parts are in place
                    if (later) bulk_wait();
                    else bulk_wait_read();
                    __syncwarp();
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        *reinterpret_cast<uint4*>(sg + tc::sw128_off(lane, i)) =
                            make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
                    tc::fence_async_smem();
                    __syncwarp();
                    if (n0 < a.N) {
                        if (add && a.out_f32) tma_add_3d(one, &p.tmo, so, t.col0 + c, n0, t.g);
                        else tma_store_3d(one, &p.tmo, so, t.col0 + c, n0, t.g);
                        bulk_commit();
                    }
                }
                if (empty) break;
                tc::tc_fence_before();
                __syncwarp();
                if (lane == 0) release(&bar_free[buf]);
                ++acc;
                p0 += part;
            }
        }
        if (kDir == kGmmDw) bulk_wait();  // the last boxes are read (and written) before the block ends
    }
    __syncwarp();
    if constexpr (kSplit) {
        // Every block adds up its share of the columns, in the blocks' order: eight columns of a row a thread and step.
        cluster_arrive();
        cluster_wait();
        const int tile = blockIdx.x / team, g = tile / p.real, in = tile % p.real;
        const int n = in / p.across * kLanes + tid % kLanes, col0 = in % p.across * kCols, share = kCols / team;
        const int c1 = min((sched.share + 1) * share, a.K - col0);
        if (tid < 2 * kLanes && n < a.N)
            for (int c = sched.share * share + tid / kLanes * 8; c < c1; c += 16) {
                float f[8] = {};
                for (int b = 0; b < team; ++b)
#pragma unroll
                    for (int j = 0; j < 8; ++j) f[j] += ld_of(sbase + ((c + j) * kLanes + tid % kLanes) * 4, b);
                const int64_t at = ((int64_t)g * a.N + n) * a.K + col0 + c;
                if (a.out_f32) {
                    float4* o = reinterpret_cast<float4*>(reinterpret_cast<float*>(a.out) + at);
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const float4 old = a.accumulate ? o[h] : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                        o[h] = make_float4(old.x + f[4 * h], old.y + f[4 * h + 1], old.z + f[4 * h + 2], old.w + f[4 * h + 3]);
                    }
                } else {
                    uint4* o = reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(a.out) + at);
                    if (a.accumulate) {
                        const uint4 old = *o;
                        const uint32_t e[4] = {old.x, old.y, old.z, old.w};
#pragma unroll
                        for (int j = 0; j < 8; ++j) f[j] += from16<kF16>((uint16_t)(e[j / 2] >> (j % 2 * 16)));
                    }
                    uint32_t w[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) w[j] = pack16<kF16>(__float_as_uint(f[2 * j]), __float_as_uint(f[2 * j + 1]));
                    *o = make_uint4(w[0], w[1], w[2], w[3]);
                }
            }
        __syncwarp();
        cluster_arrive(), cluster_wait();  // (no block ends while another reads it: the reads come before this arrival)
    }
    if (kCta == 2) cluster_arrive_relaxed(), cluster_wait();  // (neither block ends while the other still reaches into it)
    else __syncthreads();
    if (warp == 1) tmem_free<kCta>(tmem, 512);
}

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    if (!fn) {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult r = cudaDriverEntryPointSymbolNotFound;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &f, cudaEnableDefault, &r) == cudaSuccess &&
            r == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
    }
    return fn;
}

// Map of [outer][rows][cols] elements (outer = 0: two dimensions) in 128-byte-swizzled boxes of 128 bytes x box_rows;
// what lies outside reads as zero and is not written.
bool encode(CUtensorMap* m, CUtensorMapDataType type, int size, const void* base, int64_t cols, int64_t rows,
            int64_t outer, int box_rows) {
    const cuuint64_t dims[3] = {(cuuint64_t)cols, (cuuint64_t)rows, (cuuint64_t)(outer ? outer : 1)};
    const cuuint64_t strides[2] = {(cuuint64_t)cols * size, (cuuint64_t)cols * rows * size};
    const cuuint32_t box[3] = {(cuuint32_t)(128 / size), (cuuint32_t)box_rows, 1};
    const cuuint32_t step[3] = {1, 1, 1};
    return encode_fn() && encode_fn()(m, type, outer ? 3 : 2, const_cast<void*>(base), dims, strides, box, step,
                       CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                       CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// An MN-major operand [outer][terms][cols] as [outer][cols / 64][terms][64]: a box of 64 terms and `blocks` column
// blocks lands as that many 64 x 64 boxes side by side, one request instead of `blocks`.  Needs whole blocks (else a
// row's last block would run into the next row): cols % 64 == 0.
bool encode_mn(CUtensorMap* m, CUtensorMapDataType type, const void* base, int64_t cols, int64_t terms, int64_t outer,
               int blocks) {
    const cuuint64_t dims[4] = {64, (cuuint64_t)terms, (cuuint64_t)(cols / 64), (cuuint64_t)(outer ? outer : 1)};
    const cuuint64_t strides[3] = {(cuuint64_t)cols * 2, 128, (cuuint64_t)cols * terms * 2};
    const cuuint32_t box[4] = {64, 64, (cuuint32_t)blocks, 1};
    const cuuint32_t step[4] = {1, 1, 1, 1};
    return encode_fn() && encode_fn()(m, type, outer ? 4 : 3, const_cast<void*>(base), dims, strides, box, step,
                       CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                       CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int kDir, int kF16, int kCta, int kNarrow, int kSplit = 0>
cudaError_t launch_cta(const TcGmm& p, int64_t tiles, cudaStream_t s) {
    constexpr size_t smem = Ring<kDir, kCta, kNarrow>::smem;
    constexpr auto kernel = gmm_tc_kernel<kDir, kF16, kCta, kNarrow, kSplit>;
    using R = Ring<kDir, kCta, kNarrow>;
    static_assert(!kSplit || (kDir == kGmmDw && kCols * kLanes * 4 <= R::stages * R::bytes), "sums take the operands' place");
    static SmemLimit limit;
    const cudaError_t e = limit.raise((const void*)kernel, smem);
    if (e != cudaSuccess) return e;
    if (kSplit) return launch_dependent(kernel, dim3((unsigned)tiles * p.a.splits), kThreads, smem, p.a.splits, s, p);
    return launch_dependent(kernel, dim3((unsigned)std::min<int64_t>(tiles, device_sms() / kCta) * kCta), kThreads, smem,
                            kCta, s, p);
}

template <int kDir, int kF16>
cudaError_t launch_dir(const TcGmm& p, int pair, int64_t tiles, cudaStream_t s) {
    if constexpr (kDir != kGmmDw)
        if (pair)
            return p.a.M <= kNarrowRows ? launch_cta<kDir, kF16, 2, 1>(p, tiles, s) : launch_cta<kDir, kF16, 2, 0>(p, tiles, s);
    if constexpr (kDir == kGmmDw)
        if (p.a.splits > 1) return launch_cta<kDir, kF16, 1, 0, 1>(p, tiles, s);
    return launch_cta<kDir, kF16, 1, 0>(p, tiles, s);
}

inline bool on16(const void* p) { return ((uintptr_t)p & 15) == 0; }

}  // namespace

// TMA needs 16-byte aligned bases and row pitches (multiples of 8 elements) for what it reads, and for the weight
// gradient that it writes.
bool grouped_tc_supported(int dir, const GmmArgs& a) {
    if (!on16(a.a) || !on16(a.b) || a.K % 8 || !encode_fn()) return false;
    if (dir != kGmmFwd && a.N % 8) return false;
    return dir != kGmmDw || on16(a.out);
}

int64_t grouped_tc_tiles(int64_t M, int64_t J, int* at_once) {
    const int pair = J > kLanes;
    *at_once = device_sms() >> pair;
    return (J + (kLanes << pair) - 1) / (kLanes << pair) * ((M + kCols - 1) / kCols);
}

cudaError_t launch_grouped_tc(int dir, int f16, const GmmArgs& a, int pitch, cudaStream_t s) {
    TcGmm p;
    p.a = a;
    const CUtensorMapDataType t = f16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    const int64_t J = dir == kGmmDx ? a.K : a.N;  // the lanes' side
    const int pair = dir != kGmmDw && J > kLanes, per = kLanes << pair;
    int64_t tiles = (J + per - 1) / per;
    bool ok;
    p.wide_a = dir == kGmmDx ? a.K % 64 == 0 : dir == kGmmDw && a.N % 64 == 0;
    p.wide_b = dir == kGmmDw && a.K % 64 == 0;
    if (dir == kGmmDw) {
        ok = (p.wide_a ? encode_mn(&p.tma, t, a.a, a.N, a.M, 0, 2) : encode(&p.tma, t, 2, a.a, a.N, a.M, 0, 64)) &&
             (p.wide_b ? encode_mn(&p.tmb[0], t, a.b, a.K, a.M, 0, kCols / 64) : encode(&p.tmb[0], t, 2, a.b, a.K, a.M, 0, 64)) &&
             encode(&p.tmo, a.out_f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : t, a.out_f32 ? 4 : 2, a.out, a.K, a.N, a.G,
                    32);
        p.across = (a.K + kCols - 1) / kCols;
        p.real = (int)tiles * p.across;
        tiles = (int64_t)a.G * p.real;
        // Few tiles and many rows (adapter factors): as many blocks as would be idle, up to eight, share a tile's rows, at
        // least two steps of the average group's each (16384 rows, one group, 16 x 2048, fp32: 27 us, one block a tile 91;
        // 6712 rows, 3 groups of 64 x 88: 8.5 and 19.7; 1024 rows, 16 x 2048: 9.5 and 9.9).
        int splits = 8;
        while (splits > 1 && (tiles * splits > device_sms() || a.M / a.G < 2 * kStep * splits)) splits /= 2;
        p.a.splits = splits;
    } else {
        const int64_t terms = pitch ? pitch : dir == kGmmFwd ? a.K : a.N;
        ok = p.wide_a ? encode_mn(&p.tma, t, a.b, a.K, a.N, a.G, 2)
                      : encode(&p.tma, t, 2, a.b, a.K, a.N, a.G, dir == kGmmFwd ? kLanes : 64);
        // the boxes that a tile of so few rows may need (each costs the caller 0.1 us)
        const int unit = kCols / kBoxes >> pair;
        for (int i = 0; i < kBoxes && (i == 0 || (i * unit << pair) < a.M); ++i)
            ok = ok && encode(&p.tmb[i], t, 2, a.a, terms, a.M, 0, (i + 1) * unit);
        p.real = (int)tiles;
        p.across = p.real * std::max(a.splits, 1);
        tiles = p.across * (a.M / kCols + (a.off ? (int64_t)a.G : 1));
    }
    p.inv_real = 1.0f / (float)p.real;
    p.inv = 1.0f / (float)p.across;
    p.table = dir != kGmmDw && a.off && a.G <= kTable && tiles < (1 << 30);
    if (!ok) return cudaErrorInvalidValue;
    switch (dir) {
        case kGmmFwd: return f16 ? launch_dir<kGmmFwd, 1>(p, pair, tiles, s) : launch_dir<kGmmFwd, 0>(p, pair, tiles, s);
        case kGmmDx: return f16 ? launch_dir<kGmmDx, 1>(p, pair, tiles, s) : launch_dir<kGmmDx, 0>(p, pair, tiles, s);
        default: return f16 ? launch_dir<kGmmDw, 1>(p, pair, tiles, s) : launch_dir<kGmmDw, 0>(p, pair, tiles, s);
    }
}

}  // namespace moeq
