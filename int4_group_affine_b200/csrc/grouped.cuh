// grouped.cuh - products grouped by expert with ragged sizes: the arguments the launchers
// share, and how a warp finds a tile's group from the offsets.
#pragma once

#include "common.cuh"

namespace moeq {

// What a product sums over and yields, for rows m of group g (W [G][N][K]):
//   kGmmFwd: y[m][n]    = sum_k x[m][k] W[g][n][k]
//   kGmmDx:  dx[m][k]   = sum_n dy[m][n] W[g][n][k]
//   kGmmDw:  dw[g][n][k] = sum_m dy[m][n] x[m][k]
enum GmmDir { kGmmFwd = 0, kGmmDx = 1, kGmmDw = 2 };

struct GmmArgs {
    const uint16_t* a;   // x (fwd), dy (dx, dw)
    const uint16_t* b;   // W (fwd, dx), x (dw)
    const int32_t* off;  // device [G+1], or NULL: one group of all M rows
    void* out;
    int M, G, N, K;
    int out_f32;         // dw: fp32 output instead of the inputs' type
    int accumulate;      // dw: out += instead of out =
    // dw: blocks that share a tile's rows (the launchers set it); forward and dx of one group without offsets: the sum in
    // `splits` parts of `per` terms (a multiple of 64), each written as fp32 [splits][M][outputs] to `partial` instead of
    // `out`; splits <= 1: not split
    int splits, per;
    float* partial;
    int32_t* status;
    uint64_t wait_ns;
};

// The tcgen05 kernel (grouped_tc.cu), and whether it takes these operands.
bool grouped_tc_supported(int dir, const GmmArgs& a);
// `pitch`: elements from one row of a.a to the next (0: as many as the sum has terms).
cudaError_t launch_grouped_tc(int dir, int f16, const GmmArgs& a, int pitch, cudaStream_t s);
// Tiles of one group of M rows by J outputs there, and how many run at once.
int64_t grouped_tc_tiles(int64_t M, int64_t J, int* at_once);

// A group's rows.  The device sees the offsets for the first time, so whatever they hold no row
// may be touched out of range or by two groups: they are clamped to [0, M] and a running maximum
// makes them non-decreasing (which changes nothing for a proper prefix sum).
struct GmmRows {
    int begin, end;
};

__device__ __forceinline__ int gmm_clamped(const GmmArgs& a, int g) { return min(max(ld_after(a.off + g), 0), a.M); }

// The rows of group g (a whole warp; the result is the same in every lane).
__device__ __forceinline__ GmmRows gmm_rows_of(const GmmArgs& a, int g, int lane) {
    if (!a.off) return GmmRows{0, a.M};
    int m = 0;
    for (int i = lane; i <= g; i += 32) m = max(m, gmm_clamped(a, i));
    const int begin = __reduce_max_sync(0xffffffffu, m);
    return GmmRows{begin, max(begin, gmm_clamped(a, g + 1))};
}

// Walks the groups in order, 32 at a time, for a warp whose tile indices only grow: every group
// with `count` rows owns ceil(count / tile_rows) * tiles_across tiles.
struct GmmWalk {
    int g0 = 0;             // first group of the window
    int64_t before = 0;     // tiles of the groups before it
    int top = 0;            // running maximum of the offsets before it
    int begin, end;         // this lane's group
    int64_t upto;           // tiles up to and with this lane's group
    bool loaded = false;

    __device__ __forceinline__ void load(const GmmArgs& a, int lane, int tile_rows, int tiles_across) {
        const int g = g0 + lane;
        if (!a.off) {
            begin = 0;
            end = g == 0 ? a.M : 0;
        } else {
            int b = g <= a.G ? gmm_clamped(a, g) : 0, e = g < a.G ? gmm_clamped(a, g + 1) : 0;
            b = max(b, top);
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(0xffffffffu, b, o);
                if (lane >= o) b = max(b, v);
            }
            begin = b;
            end = g < a.G ? max(b, e) : b;
        }
        const int count = g < a.G ? end - begin : 0;
        int64_t t = (int64_t)((count + tile_rows - 1) / tile_rows) * tiles_across;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t v = __shfl_up_sync(0xffffffffu, t, o);
            if (lane >= o) t += v;
        }
        upto = before + t;
        loaded = true;
    }

    // The group that owns `tile` (-1: no group does), its rows and the tile's index within it.
    __device__ __forceinline__ int find(const GmmArgs& a, int lane, int64_t tile, int tile_rows, int tiles_across,
                                        GmmRows* rows, int64_t* within) {
        if (!loaded) load(a, lane, tile_rows, tiles_across);
        for (;;) {
            const uint32_t past = __ballot_sync(0xffffffffu, tile < upto);
            if (past) {
                const int l = __ffs(past) - 1;
                const int64_t prev = __shfl_sync(0xffffffffu, upto, l > 0 ? l - 1 : 0);
                rows->begin = __shfl_sync(0xffffffffu, begin, l);
                rows->end = __shfl_sync(0xffffffffu, end, l);
                *within = tile - (l > 0 ? prev : before);
                return g0 + l;
            }
            if (g0 + 32 >= a.G) return -1;
            before = __shfl_sync(0xffffffffu, upto, 31);
            top = __shfl_sync(0xffffffffu, end, 31);
            g0 += 32;
            load(a, lane, tile_rows, tiles_across);
        }
    }
};

// Whether this thread's share of the offsets (one block's threads, any count) is a non-decreasing sequence within
// [0, M]; the first block raises MOE_ERR_DEVICE_INDEX where it is not.
__device__ __forceinline__ bool gmm_check_offsets(const GmmArgs& a, int tid, int nthreads) {
    if (!a.off) return true;
    bool good = true;
    for (int g = tid; g <= a.G; g += nthreads) {
        const int v = ld_after(a.off + g);
        if (v < 0 || v > a.M || (g > 0 && ld_after(a.off + g - 1) > v)) good = false;
    }
    if (!good && blockIdx.x == 0) raise_status(a.status, MOE_ERR_DEVICE_INDEX);
    return good;
}

}  // namespace moeq
