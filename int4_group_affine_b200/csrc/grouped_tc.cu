// grouped_tc.cu - products grouped by expert with ragged sizes, and their gradients, on the tcgen05
// tensor cores (sm_100a): operands by TMA, accumulators in tensor memory.
//
// One persistent kernel for the three directions.  A tile of the output is 128 matrix rows (the
// tensor memory's lanes) by up to 256 columns, over the sum in steps of 64:
//
//   forward  lanes = outputs n of W[g], columns = rows m of the group, sum over k
//   dx       lanes = inputs k of W[g],  columns = rows m of the group, sum over n
//   dw       lanes = outputs n,         columns = inputs k,            sum over the group's rows m
//
// With the matrix on the lanes, the ragged side is the one whose width the instruction can choose: a
// group of c rows takes ceil(c / 256) tiles of equal width, rounded up to 16, so a group of 17 rows
// multiplies 32 columns and not 128.  An operand whose summed index is contiguous in memory (W and x
// in the forward, dy in dx) is stored K-major, the others (W in dx; dy and x in dw) MN-major: the
// 128-byte-swizzled boxes that TMA writes are the tensor core's own layout for either, so nothing is
// transposed by hand.
//
// Rows of other groups.  The row boxes run past a group's end.  In forward and dx those rows only
// fill columns that are not stored.  In dw they would enter the sum, so the MMA warp clears them in
// both operands (a NaN times zero is a NaN) up to the next 16, and multiplies no further.
//
// Warps: 0 loads (one lane issues TMA into a ring of four 48 KB stages), 1 multiplies (one lane
// issues tcgen05.mma), 2..9 write results, two per quarter of the lanes; the accumulator is double
// buffered, so a tile is written while the next one multiplies.  forward and dx: a warp stores, for
// each row m, its 32 lanes' outputs as one 64-byte piece.  dw: 32 x 128-byte boxes through shared
// memory and TMA stores, which clip at the matrix's edges.  Every wait is bounded.
//
// fp32 weight gradients: the tensor core's accumulation rounds toward zero, an error that grows with
// the sum's length (measured 4.7e-7 of the result at 512 terms, 9.1e-6 at 8192), so sums longer than
// 512 rows leave the tensor core in parts and are added by the L2's fp32 additions, one part after
// the other (a fixed order).
#include <cuda_fp16.h>
#include <cudaTypedefs.h>

#include "grouped.cuh"
#include "tc.cuh"

namespace moeq {
namespace {

constexpr int kLanes = 128;              // output tile: matrix rows
constexpr int kCols = 256;               // and at most this many columns
constexpr int kStep = 64;                // terms per stage
constexpr int kStages = 4;
constexpr int kABytes = kLanes * 128;    // 64 16-bit terms of every lane
constexpr int kBBytes = kCols * 128;
constexpr int kStageBytes = kABytes + kBBytes;
constexpr int kBox = 64 * 128;           // an MN-major box: 64 terms of 64 outputs
constexpr int kEpi = 8;                  // result warps
constexpr int kThreads = (2 + kEpi) * 32;
constexpr int kOutBytes = 32 * 128;      // dw: a warp's staging box
constexpr int kPart = 512;               // fp32 dw: terms per part
constexpr size_t kSmem = 1024 + kStages * kStageBytes + kEpi * kOutBytes;
static_assert(kSmem + 1024 <= 227 * 1024, "shared memory");

struct TcGmm {
    CUtensorMap tma;     // the lanes' operand
    CUtensorMap tmb;     // the columns' operand, in boxes of 128 rows (forward, dx) or 64 x 64 (dw)
    CUtensorMap tmb16;   // forward, dx: the same in boxes of 16 rows
    CUtensorMap tmo;     // dw: the output, in boxes of 32 rows x 128 bytes
    GmmArgs a;
};

// A tile of work as every warp role sees it.
struct Tile {
    int g;         // group (-1: no more)
    int lane0;     // first output row of the tile
    int col0;      // first column: row of x / dy (forward, dx), input k (dw)
    int cols;      // columns that count
    int width;     // columns multiplied: cols rounded up to 16
    int terms;     // length of the sum
    int row0;      // dw: first row of the group
};

template <int kDir>
struct Schedule {
    GmmWalk walk;
    int g_dw = -1;
    GmmRows rows_dw;

    __device__ __forceinline__ Tile at(const GmmArgs& a, int64_t tile, int lane) {
        Tile t;
        if (kDir == kGmmDw) {
            const int nt = (a.N + kLanes - 1) / kLanes, kt = (a.K + kCols - 1) / kCols;
            const int64_t per = (int64_t)nt * kt;
            t.g = tile < per * a.G ? (int)(tile / per) : -1;
            if (t.g < 0) return t;
            if (t.g != g_dw) rows_dw = gmm_rows_of(a, g_dw = t.g, lane);
            const int rem = (int)(tile % per);
            t.lane0 = rem / kt * kLanes;
            t.col0 = rem % kt * kCols;
            t.cols = min(kCols, a.K - t.col0);
            t.terms = rows_dw.end - rows_dw.begin;
            t.row0 = rows_dw.begin;
        } else {
            const int J = kDir == kGmmFwd ? a.N : a.K, across = (J + kLanes - 1) / kLanes;
            GmmRows r;
            int64_t within;
            t.g = walk.find(a, lane, tile, kCols, across, &r, &within);
            if (t.g < 0) return t;
            const int count = r.end - r.begin, parts = (count + kCols - 1) / kCols;
            const int w = ((count + parts - 1) / parts + 15) & ~15;
            const int p = (int)(within / across);
            t.lane0 = (int)(within % across) * kLanes;
            t.col0 = r.begin + p * w;
            t.cols = min(w, count - p * w);
            t.terms = kDir == kGmmFwd ? a.K : a.N;
        }
        t.width = (t.cols + 15) & ~15;
        return t;
    }
};

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const void* map, int x, int y, int z, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], "
        "[%5];" ::"r"(dst),
        "l"(map), "r"(x), "r"(y), "r"(z), "r"(tc::smem_u32(bar))
        : "memory");
}
__device__ __forceinline__ void tma_store_3d(const void* map, uint32_t src, int x, int y, int z) {
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(map),
                 "r"(src), "r"(x), "r"(y), "r"(z)
                 : "memory");
}
__device__ __forceinline__ void tma_add_3d(const void* map, uint32_t src, int x, int y, int z) {
    asm volatile("cp.reduce.async.bulk.tensor.3d.global.shared::cta.add.tile.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(
                     map),
                 "r"(src), "r"(x), "r"(y), "r"(z)
                 : "memory");
}
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

template <int kDir>
__device__ __forceinline__ uint32_t idesc_of(int f16, int width) {
    const uint32_t t = f16 ? 0u : 1u;
    return (1u << 4) | (t << 7) | (t << 10) | (kDir != kGmmFwd ? 1u << 15 : 0u) | (kDir == kGmmDw ? 1u << 16 : 0u) |
           ((uint32_t)(width >> 3) << 17) | ((uint32_t)(kLanes >> 4) << 24);
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
__device__ __forceinline__ uint32_t pack16(float lo, float hi) {
    return (uint32_t)to16<kF16>(lo) | ((uint32_t)to16<kF16>(hi) << 16);
}

// A whole warp's wait: the same answer in every lane, so that a wait that gives up never splits the warp.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, const GmmArgs& a, volatile int* ok) {
    return __all_sync(0xffffffffu, tc::mbar_wait_ok(bar, parity, a.status, ok, a.wait_ns));
}

template <int kDir, int kF16>
__global__ void __launch_bounds__(kThreads, 1) gmm_tc_kernel(const __grid_constant__ TcGmm p) {
    extern __shared__ unsigned char raw[];
    unsigned char* sm = raw + ((1024u - (tc::smem_u32(raw) & 1023u)) & 1023u);
    unsigned char* s_out = sm + kStages * kStageBytes;
    __shared__ uint64_t bar_full[kStages], bar_empty[kStages];  // a stage landed / was multiplied
    __shared__ uint64_t bar_acc[2], bar_free[2];                // an accumulator is complete / was read
    __shared__ uint64_t bar_drain;
    __shared__ uint32_t s_tmem;
    __shared__ volatile int s_ok;
    const GmmArgs& a = p.a;
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;

    if (warp == 1) {
        tc::tmem_alloc(&s_tmem, 512);
        tc::tmem_relinquish();
    }
    if (tid == 0) {
        for (int i = 0; i < kStages; ++i) {
            tc::mbar_init(&bar_full[i], 1);
            tc::mbar_init(&bar_empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            tc::mbar_init(&bar_acc[i], 1);
            tc::mbar_init(&bar_free[i], kEpi);
        }
        tc::mbar_init(&bar_drain, 1);
        tc::mbar_init_fence();
        s_ok = 1;
        tc::tma_prefetch_desc(&p.tma);
        tc::tma_prefetch_desc(&p.tmb);
        tc::tma_prefetch_desc(kDir == kGmmDw ? &p.tmo : &p.tmb16);
    }
    if (blockIdx.x == 0) gmm_check_offsets(a, tid, kThreads);
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    const uint32_t tmem = s_tmem;
    const uint32_t sbase = tc::smem_u32(sm);
    Schedule<kDir> sched;
    const bool parts = kDir == kGmmDw && a.out_f32;  // long sums in parts

    if (warp == 0) {
        // ------------------------------------------------------------ loads
        uint32_t n = 0;  // stages issued
        for (int64_t tile = blockIdx.x;; tile += gridDim.x) {
            const Tile t = sched.at(a, tile, lane);
            if (t.g < 0 || __any_sync(0xffffffffu, !s_ok)) break;
            if (lane == 0) {
                const int b128 = kDir == kGmmDw ? 0 : t.width / 128, b16 = kDir == kGmmDw ? 0 : t.width % 128 / 16;
                const int bk = kDir == kGmmDw ? (t.cols + 63) / 64 : 0;
                const uint32_t bytes = kABytes + b128 * 128 * 128 + b16 * 16 * 128 + bk * kBox;
                for (int k = 0; k < t.terms; k += kStep, ++n) {
                    const int st = n % kStages;
                    if (n >= kStages &&
                        !tc::mbar_wait_ok(&bar_empty[st], (n / kStages - 1) & 1, a.status, &s_ok, a.wait_ns))
                        break;
                    const uint32_t sa = sbase + st * kStageBytes, sb = sa + kABytes;
                    uint64_t* full = &bar_full[st];
                    tc::mbar_arrive_expect_tx(full, bytes);
                    if (kDir == kGmmFwd) {
                        tma_load_3d(sa, &p.tma, k, t.lane0, t.g, full);
                    } else if (kDir == kGmmDx) {
                        tma_load_3d(sa, &p.tma, t.lane0, k, t.g, full);
                        tma_load_3d(sa + kBox, &p.tma, t.lane0 + 64, k, t.g, full);
                    } else {
                        tc::tma_load_2d(sa, &p.tma, t.lane0, t.row0 + k, full);
                        tc::tma_load_2d(sa + kBox, &p.tma, t.lane0 + 64, t.row0 + k, full);
                    }
                    if (kDir == kGmmDw) {
                        for (int i = 0; i < bk; ++i)
                            tc::tma_load_2d(sb + i * kBox, &p.tmb, t.col0 + 64 * i, t.row0 + k, full);
                    } else {
                        for (int i = 0; i < b128; ++i)
                            tc::tma_load_2d(sb + i * 128 * 128, &p.tmb, k, t.col0 + 128 * i, full);
                        for (int i = 0; i < b16; ++i)
                            tc::tma_load_2d(sb + b128 * 128 * 128 + i * 16 * 128, &p.tmb16, k,
                                            t.col0 + 128 * b128 + 16 * i, full);
                    }
                }
            }
            __syncwarp();
        }
        if (lane == 0 && !s_ok)  // given up: wait for the copies still in flight before the block ends
            for (uint32_t i = n > kStages ? n - kStages : 0; i < n; ++i)
                tc::mbar_wait(&bar_full[i % kStages], (i / kStages) & 1, a.status, a.wait_ns);
    } else if (warp == 1) {
        // ------------------------------------------------------------ products
        uint32_t n = 0, acc = 0;
        bool ok = true;
        for (int64_t tile = blockIdx.x; ok; tile += gridDim.x) {
            const Tile t = sched.at(a, tile, lane);
            if (t.g < 0) break;
            const uint32_t idesc = idesc_of<kDir>(kF16, t.width);
            for (int p0 = 0; ok && p0 < t.terms; ++acc) {
                const int p1 = parts ? min(t.terms, p0 + kPart) : t.terms;
                const uint32_t d = tmem + (acc & 1) * kCols;
                if (acc >= 2) ok = warp_wait(&bar_free[acc & 1], (acc / 2 - 1) & 1, a, &s_ok);
                tc::tc_fence_after();
                for (int k = p0; ok && k < p1; k += kStep, ++n) {
                    const int st = n % kStages;
                    ok = warp_wait(&bar_full[st], (n / kStages) & 1, a, &s_ok);
                    if (!ok) break;
                    const uint32_t sa = sbase + st * kStageBytes, sb = sa + kABytes;
                    const int left = min(kStep, t.terms - k), m16 = (left + 15) / 16;
                    if (kDir == kGmmDw && left % 16) {  // the rows behind the group's last, up to the next 16
                        const int clear = (m16 * 16 - left) * 8, bk = (t.cols + 63) / 64;
                        unsigned char* base = sm + st * kStageBytes + left * 128;
                        for (int b = 0; b < 2 + bk; ++b)
                            for (int i = lane; i < clear; i += 32)
                                *reinterpret_cast<uint4*>(base + b * kBox + i * 16) = make_uint4(0, 0, 0, 0);
                        tc::fence_async_smem();
                        __syncwarp();
                    }
                    if (lane == 0) {
                        tc::tc_fence_after();
                        for (int s = 0; s < m16; ++s) {
                            const uint64_t ad = kDir == kGmmFwd ? tc::sdesc_k_sw128(sa + 32 * s)
                                                                : sdesc_mn_sw128(sa + 2048 * s);
                            const uint64_t bd = kDir == kGmmDw ? sdesc_mn_sw128(sb + 2048 * s)
                                                               : tc::sdesc_k_sw128(sb + 32 * s);
                            tc::mma_bf16(d, ad, bd, idesc, k > p0 || s > 0);
                        }
                        tc::mma_commit(&bar_empty[st]);
                    }
                    __syncwarp();
                }
                if (ok && lane == 0) tc::mma_commit(&bar_acc[acc & 1]);
                __syncwarp();
                p0 = p1;
            }
        }
        if (!ok && lane == 0) {  // given up: the products still in flight end before their memory is freed
            tc::mma_commit(&bar_drain);
            tc::mbar_wait(&bar_drain, 0, a.status, a.wait_ns);
        }
    } else {
        // ------------------------------------------------------------ results
        const int q = warp % 4, half = (warp - 2) / 4;  // lanes [32 q, 32 q + 32), every other piece of columns
        uint32_t acc = 0;
        bool ok = true;
        const uint32_t so = tc::smem_u32(s_out + (warp - 2) * kOutBytes);
        unsigned char* sg = s_out + (warp - 2) * kOutBytes;
        for (int64_t tile = blockIdx.x; ok; tile += gridDim.x) {
            const Tile t = sched.at(a, tile, lane);
            if (t.g < 0) break;
            if (kDir != kGmmDw) {
                ok = warp_wait(&bar_acc[acc & 1], (acc / 2) & 1, a, &s_ok);
                if (!ok) break;
                tc::tc_fence_after();
                const int J = kDir == kGmmFwd ? a.N : a.K, f = t.lane0 + 32 * q + lane;
                uint16_t* out = reinterpret_cast<uint16_t*>(a.out) + (int64_t)t.col0 * J + f;
                for (int c = 32 * half; c < t.cols; c += 64) {
                    uint32_t v[32];
                    tmem_ld32(tmem + ((uint32_t)(32 * q) << 16) + (acc & 1) * kCols + c, v);
                    tc::tmem_wait_ld();
                    const int live = f < J ? t.cols - c : 0;
                    uint16_t* o = out + (int64_t)c * J;
#pragma unroll
                    for (int i = 0; i < 32; ++i) {
                        if (i < live) *o = to16<kF16>(__uint_as_float(v[i]));
                        o += J;
                    }
                }
                tc::tc_fence_before();
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(&bar_free[acc & 1]);
                ++acc;
                continue;
            }
            // dw: pieces of 128 bytes of every lane's row (32 fp32 or 64 16-bit columns)
            const int n = t.lane0 + 32 * q + lane;
            const int per = a.out_f32 ? 32 : 64;
            const bool empty = t.terms == 0;
            if (empty && a.accumulate) continue;
            for (int p0 = 0; ok && (p0 < t.terms || empty);) {
                const bool add = a.accumulate || p0 > 0;
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
                        tmem_ld32(tmem + ((uint32_t)(32 * q) << 16) + buf * kCols + c, w);
                        tc::tmem_wait_ld();
                    } else {
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            uint32_t v[32];
                            tmem_ld32(tmem + ((uint32_t)(32 * q) << 16) + buf * kCols + c + 32 * h, v);
                            tc::tmem_wait_ld();
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
                                w[16 * h + i] = pack16<kF16>(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1]));
                        }
                    }
                    if (lane == 0) {  // the staging box is free, and earlier parts are in place
                        if (p0 > 0) bulk_wait();
                        else bulk_wait_read();
                    }
                    __syncwarp();
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        *reinterpret_cast<uint4*>(sg + tc::sw128_off(lane, i)) =
                            make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
                    tc::fence_async_smem();
                    __syncwarp();
                    if (lane == 0 && t.lane0 + 32 * q < a.N) {
                        if (add && a.out_f32) tma_add_3d(&p.tmo, so, t.col0 + c, t.lane0 + 32 * q, t.g);
                        else tma_store_3d(&p.tmo, so, t.col0 + c, t.lane0 + 32 * q, t.g);
                        bulk_commit();
                    }
                }
                if (empty) break;
                tc::tc_fence_before();
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(&bar_free[buf]);
                ++acc;
                p0 = parts ? p0 + kPart : t.terms;
            }
        }
        if (kDir == kGmmDw && lane == 0) bulk_wait();  // the last boxes are read (and written) before the block ends
    }
    __syncthreads();
    if (warp == 1) tc::tmem_dealloc(tmem, 512);
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
    return encode_fn()(m, type, outer ? 3 : 2, const_cast<void*>(base), dims, strides, box, step,
                       CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                       CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int kDir, int kF16>
cudaError_t launch_dir(const TcGmm& p, int64_t tiles, cudaStream_t s) {
    int dev = 0, nsm = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&nsm, cudaDevAttrMultiProcessorCount, dev);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute((const void*)gmm_tc_kernel<kDir, kF16>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 (int)kSmem);
    if (e != cudaSuccess) return e;
    gmm_tc_kernel<kDir, kF16><<<(unsigned)(tiles < nsm ? tiles : nsm), kThreads, kSmem, s>>>(p);
    return cudaGetLastError();
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

cudaError_t launch_grouped_tc(int dir, int f16, const GmmArgs& a, cudaStream_t s) {
    TcGmm p;
    p.a = a;
    const CUtensorMapDataType t = f16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    const int64_t nt = (a.N + kLanes - 1) / kLanes;
    int64_t tiles;
    bool ok;
    if (dir == kGmmDw) {
        ok = encode(&p.tma, t, 2, a.a, a.N, a.M, 0, 64) && encode(&p.tmb, t, 2, a.b, a.K, a.M, 0, 64) &&
             encode(&p.tmo, a.out_f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : t, a.out_f32 ? 4 : 2, a.out, a.K, a.N, a.G,
                    32);
        p.tmb16 = p.tmb;
        tiles = a.G * nt * ((a.K + kCols - 1) / kCols);
    } else {
        const int64_t terms = dir == kGmmFwd ? a.K : a.N;
        ok = encode(&p.tma, t, 2, a.b, a.K, a.N, a.G, dir == kGmmFwd ? kLanes : 64) &&
             encode(&p.tmb, t, 2, a.a, terms, a.M, 0, 128) && encode(&p.tmb16, t, 2, a.a, terms, a.M, 0, 16);
        p.tmo = p.tmb;
        tiles = (a.M / kCols + (a.off ? (int64_t)a.G : 1)) * (dir == kGmmFwd ? nt : (a.K + kLanes - 1) / kLanes);
    }
    if (!ok) return cudaErrorInvalidValue;
    switch (dir) {
        case kGmmFwd: return f16 ? launch_dir<kGmmFwd, 1>(p, tiles, s) : launch_dir<kGmmFwd, 0>(p, tiles, s);
        case kGmmDx: return f16 ? launch_dir<kGmmDx, 1>(p, tiles, s) : launch_dir<kGmmDx, 0>(p, tiles, s);
        default: return f16 ? launch_dir<kGmmDw, 1>(p, tiles, s) : launch_dir<kGmmDw, 0>(p, tiles, s);
    }
}

}  // namespace moeq
