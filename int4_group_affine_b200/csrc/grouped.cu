// grouped.cu - products grouped by expert with ragged sizes, and their gradients, on warp-level
// tensor-core tiles: the kernel that takes every size, alignment and row count.
//
// A block owns a 64 x 64 tile of the output and steps through the sum 32 terms at a time: both
// operands come into shared memory by guarded 2-byte loads (zero outside the matrix and, for the
// weight gradient, outside the group's rows, so a NaN in another group's row never meets a sum),
// laid out [row][term] with an 80-byte pitch (the eight rows a fragment load touches start 20 banks
// apart: no two of its 32 words share a bank), and four warps of 32 x 32 run mma.sync m16n8k16 with
// fp32 accumulators.  The loads follow the operand's contiguous axis, so they coalesce in all three
// directions.
#include <cuda_fp16.h>

#include "grouped.cuh"

namespace moeq {
namespace {

constexpr int kT = 64, kKT = 32, kPitch = 40, kThreads = 128;
// fp32 results: the tensor core's fp32 accumulation rounds toward zero, an error that grows with
// the length of the sum (measured 4.7e-7 of the result at 512 terms, 9.1e-6 at 8192); sums longer
// than this are added up in parts of this length with rounded fp32 additions.
constexpr int kPart = 512;

template <int kF16>
__device__ __forceinline__ void mma16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if (kF16)
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, "
            "%2, %3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, "
            "%1, %2, %3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <int kF16>
__device__ __forceinline__ uint16_t to16(float v) {
    return kF16 ? __half_as_ushort(__float2half_rn(v)) : f2bf16(v);
}
template <int kF16>
__device__ __forceinline__ float from16(uint16_t v) {
    return kF16 ? __half2float(__ushort_as_half(v)) : bf16f(v);
}

// One operand tile [64 rows][32 terms] into shared memory.  kAlong: 0 the terms are contiguous in
// memory (row stride ld), 1 the rows are (term stride ld).
template <int kAlong>
__device__ __forceinline__ void load_tile(uint16_t (*s)[kPitch], const uint16_t* __restrict__ p, int64_t ld, int r0,
                                          int rows, int t0, int terms, int tid) {
    if (kAlong == 0) {
        const int t = tid % kKT;
#pragma unroll
        for (int r = tid / kKT; r < kT; r += kThreads / kKT)
            s[r][t] = (r0 + r < rows && t0 + t < terms) ? __ldg(p + (int64_t)(r0 + r) * ld + t0 + t) : (uint16_t)0;
    } else {
        const int r = tid % kT;
#pragma unroll
        for (int t = tid / kT; t < kKT; t += kThreads / kT)
            s[r][t] = (r0 + r < rows && t0 + t < terms) ? __ldg(p + (int64_t)(t0 + t) * ld + r0 + r) : (uint16_t)0;
    }
}

template <int kDir, int kF16>
__global__ void __launch_bounds__(kThreads) gmm_any_kernel(const GmmArgs a) {
    __shared__ __align__(16) uint16_t sA[kT][kPitch], sB[kT][kPitch];
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32, g8 = lane / 4, c4 = lane % 4;
    grid_wait();
    if (blockIdx.x == 0) (void)gmm_check_offsets(a, tid, kThreads);

    // the tile: group, output rows [i0, I) and columns [j0, J), terms [0, S)
    const int J = kDir == kGmmFwd ? a.N : a.K;
    const int jt = (J + kT - 1) / kT;
    int g, i0, j0, I, S;
    GmmRows rows;
    if (kDir == kGmmDw) {
        const int it = (a.N + kT - 1) / kT;
        g = (int)(blockIdx.x / ((int64_t)it * jt));
        const int rem = (int)(blockIdx.x % ((int64_t)it * jt));
        rows = gmm_rows_of(a, g, lane);
        i0 = rem / jt * kT;
        j0 = rem % jt * kT;
        I = a.N;
        S = rows.end - rows.begin;
    } else {
        GmmWalk w;
        int64_t within;
        g = w.find(a, lane, blockIdx.x, kT, jt, &rows, &within);
        if (g < 0) return;
        i0 = (int)(within / jt) * kT;
        j0 = (int)(within % jt) * kT;
        I = rows.end - rows.begin;
        S = kDir == kGmmFwd ? a.K : a.N;
    }
    const int64_t nk = (int64_t)a.N * a.K;
    const uint16_t* pa = kDir == kGmmDw ? a.a + (int64_t)rows.begin * a.N : a.a + (int64_t)rows.begin * S;
    const uint16_t* pb = kDir == kGmmDw ? a.b + (int64_t)rows.begin * a.K : a.b + g * nk;

    float acc[2][4][4], sum[2][4][4];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int q = 0; q < 4; ++q) acc[i][j][q] = sum[i][j][q] = 0.0f;

    const int wi = warp / 2 * 32, wj = warp % 2 * 32;
    for (int t0 = 0; t0 < S; t0 += kKT) {
        __syncthreads();
        load_tile<kDir == kGmmDw>(sA, pa, kDir == kGmmDw ? a.N : S, i0, I, t0, S, tid);
        load_tile<kDir != kGmmFwd>(sB, pb, a.K, j0, J, t0, S, tid);
        __syncthreads();
#pragma unroll
        for (int ks = 0; ks < kKT; ks += 16) {
            uint32_t fa[2][4];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int r = wi + 16 * i + g8, k = ks + 2 * c4;
                fa[i][0] = *reinterpret_cast<const uint32_t*>(&sA[r][k]);
                fa[i][1] = *reinterpret_cast<const uint32_t*>(&sA[r + 8][k]);
                fa[i][2] = *reinterpret_cast<const uint32_t*>(&sA[r][k + 8]);
                fa[i][3] = *reinterpret_cast<const uint32_t*>(&sA[r + 8][k + 8]);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int r = wj + 8 * j + g8, k = ks + 2 * c4;
                const uint32_t b0 = *reinterpret_cast<const uint32_t*>(&sB[r][k]);
                const uint32_t b1 = *reinterpret_cast<const uint32_t*>(&sB[r][k + 8]);
                mma16<kF16>(acc[0][j], fa[0], b0, b1);
                mma16<kF16>(acc[1][j], fa[1], b0, b1);
            }
        }
        if ((t0 + kKT) % kPart == 0 || t0 + kKT >= S) {
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j)
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        sum[i][j][q] += acc[i][j][q];
                        acc[i][j][q] = 0.0f;
                    }
        }
    }

    const int64_t out0 = kDir == kGmmDw ? g * nk : (int64_t)rows.begin * J;
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int r = i0 + wi + 16 * i + g8 + 8 * (q / 2), c = j0 + wj + 8 * j + 2 * c4 + q % 2;
                if (r >= I || c >= J) continue;
                const int64_t at = out0 + (int64_t)r * J + c;
                float v = sum[i][j][q];
                if (kDir == kGmmDw && a.out_f32) {
                    float* o = reinterpret_cast<float*>(a.out) + at;
                    *o = a.accumulate ? *o + v : v;
                } else {
                    uint16_t* o = reinterpret_cast<uint16_t*>(a.out) + at;
                    if (kDir == kGmmDw && a.accumulate) v += from16<kF16>(*o);
                    *o = to16<kF16>(v);
                }
            }
}

template <int kDir>
cudaError_t launch_any(const GmmArgs& a, int f16, cudaStream_t s) {
    const int64_t jt = ((kDir == kGmmFwd ? a.N : a.K) + kT - 1) / kT;
    // forward and dx: a group's last tile may be partly filled, so at most one more per group
    const int64_t tiles = kDir == kGmmDw ? (int64_t)a.G * ((a.N + kT - 1) / kT) * jt
                                         : ((int64_t)a.M / kT + (a.off ? a.G : 1)) * jt;
    if (tiles > INT32_MAX) return cudaErrorInvalidConfiguration;
    return launch_dependent(f16 ? gmm_any_kernel<kDir, 1> : gmm_any_kernel<kDir, 0>, dim3((unsigned)tiles), kThreads, 0, 1, s,
                            a);
}

}  // namespace

cudaError_t launch_grouped(int dir, int f16, const GmmArgs& a, cudaStream_t s) {
    if (grouped_tc_supported(dir, a)) return launch_grouped_tc(dir, f16, a, s);
    switch (dir) {
        case kGmmFwd: return launch_any<kGmmFwd>(a, f16, s);
        case kGmmDx: return launch_any<kGmmDx>(a, f16, s);
        default: return launch_any<kGmmDw>(a, f16, s);
    }
}

}  // namespace moeq
