// linear.cu - rows times an affine-packed matrix (4 or 8 bits, groups along the input), and the
// matrix itself in bf16 for the products that go over many rows.
//
// y[t][n] = sum over groups of s * (sum q x) + b * (sum x): the codes stay whole numbers inside a
// group's sum, scale and bias come once per group.
#include "common.cuh"

namespace moeq {
namespace {

// One warp per output row and eight tokens.
template <int kBits>
__global__ void __launch_bounds__(256) linear_rows_kernel(const moe_qtensor W, const uint16_t* __restrict__ x, int T,
                                                          uint16_t* __restrict__ y) {
    constexpr int kPer = 32 / kBits;
    const int lane = threadIdx.x % 32, n = blockIdx.x * 8 + threadIdx.x / 32, t0 = blockIdx.y * 8;
    if (n >= W.out) return;
    const int words = W.in / kPer, groups = W.in / W.group;
    const uint32_t* wr = W.packed + (int64_t)n * words;
    const uint16_t *sr = W.scales + (int64_t)n * groups, *br = W.biases + (int64_t)n * groups;
    float acc[8];
#pragma unroll
    for (int t = 0; t < 8; ++t) acc[t] = 0.0f;
    for (int i = lane; i < words; i += 32) {
        const uint32_t w = __ldg(wr + i);
        const int g = i * kPer / W.group;
        const float s = bf16f(__ldg(sr + g)), b = bf16f(__ldg(br + g));
#pragma unroll
        for (int t = 0; t < 8; ++t) {
            if (t0 + t >= T) break;
            const uint16_t* xr = x + (int64_t)(t0 + t) * W.in + i * kPer;
            float qx = 0.0f, sx = 0.0f;
#pragma unroll
            for (int j = 0; j < kPer; ++j) {
                const float v = bf16f(__ldg(xr + j));
                qx = fmaf((float)((w >> (j * kBits)) & ((1u << kBits) - 1u)), v, qx);
                sx += v;
            }
            acc[t] += s * qx + b * sx;
        }
    }
#pragma unroll
    for (int t = 0; t < 8; ++t) {
        const float v = warp_sum(acc[t]);
        if (lane == 0 && t0 + t < T) y[(int64_t)(t0 + t) * W.out + n] = f2bf16(v);
    }
}

// bf16(s q + b), one thread per word.
template <int kBits>
__global__ void __launch_bounds__(256) dequant16_kernel(const moe_qtensor W, int64_t words, uint16_t* __restrict__ out) {
    constexpr int kPer = 32 / kBits;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < words; i += (int64_t)gridDim.x * 256) {
        const uint32_t w = __ldg(W.packed + i);
        const int64_t g = i * kPer / W.group;  // (a row is a whole number of groups)
        const float s = bf16f(__ldg(W.scales + g)), b = bf16f(__ldg(W.biases + g));
#pragma unroll
        for (int j = 0; j < kPer; ++j)
            out[i * kPer + j] = f2bf16(fmaf(s, (float)((w >> (j * kBits)) & ((1u << kBits) - 1u)), b));
    }
}

}  // namespace

cudaError_t launch_affine_linear(const moe_qtensor& W, const uint16_t* x, int T, uint16_t* y, cudaStream_t s) {
    const dim3 grid((W.out + 7) / 8, (T + 7) / 8);
    if (W.bits == 4) linear_rows_kernel<4><<<grid, 256, 0, s>>>(W, x, T, y);
    else linear_rows_kernel<8><<<grid, 256, 0, s>>>(W, x, T, y);
    return cudaGetLastError();
}

cudaError_t launch_affine_dequant16(const moe_qtensor& W, uint16_t* out, cudaStream_t s) {
    const int64_t words = (int64_t)W.out * W.in * W.bits / 32, want = (words + 255) / 256;
    const unsigned blocks = (unsigned)(want < 148 * 8 ? want : 148 * 8);
    if (W.bits == 4) dequant16_kernel<4><<<blocks, 256, 0, s>>>(W, words, out);
    else dequant16_kernel<8><<<blocks, 256, 0, s>>>(W, words, out);
    return cudaGetLastError();
}

}  // namespace moeq
