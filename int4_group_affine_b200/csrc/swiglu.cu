// swiglu.cu - h = w silu(gate) up on stacked [gate | up] rows with a weight per row, and its
// gradient.  The rows behind the last group are neither read nor written.
//
// With s = sigmoid(gate): d gate = w dh up s (1 + gate (1 - s)), d up = w dh gate s,
// d w = sum over the row of dh gate s up.
#include <cuda_fp16.h>

#include "common.cuh"

namespace moeq {
namespace {

template <int kF16>
__device__ __forceinline__ float ld16(uint16_t v) {
    return kF16 ? __half2float(__ushort_as_half(v)) : bf16f(v);
}
template <int kF16>
__device__ __forceinline__ uint16_t st16(float v) {
    return kF16 ? __half_as_ushort(__float2half_rn(v)) : f2bf16(v);
}

struct Range {
    int begin, end;
};
__device__ __forceinline__ Range rows_of(const SwigluArgs& a) {
    if (!a.off) return Range{0, a.M};
    return Range{max(__ldg(a.off), 0), min(__ldg(a.off + a.G), a.M)};
}

// One block per row.
template <int kF16, int kGrad>
__global__ void __launch_bounds__(256) swiglu_kernel(const SwigluArgs a) {
    __shared__ float s_part[8];
    const Range r = rows_of(a);
    const int64_t m = blockIdx.x;
    if (m < r.begin || m >= r.end) return;
    const int I = a.I;
    const uint16_t *gr = a.gu + m * 2 * I, *ur = gr + I;
    const float w = a.w ? __ldg(a.w + m) : 1.0f;
    float dw = 0.0f;
    for (int i = threadIdx.x; i < I; i += 256) {
        const float g = ld16<kF16>(__ldg(gr + i)), u = ld16<kF16>(__ldg(ur + i));
        const float s = 1.0f / (1.0f + expf(-g)), sl = g * s;
        if (!kGrad) {
            a.h[m * I + i] = st16<kF16>(w * sl * u);
        } else {
            const float d = ld16<kF16>(__ldg(a.dh + m * I + i));
            a.dgu[m * 2 * I + i] = st16<kF16>(w * d * u * s * (1.0f + g * (1.0f - s)));
            a.dgu[m * 2 * I + I + i] = st16<kF16>(w * d * sl);
            dw = fmaf(d, sl * u, dw);
        }
    }
    if (kGrad && a.dw) {
        dw = warp_sum(dw);
        if (threadIdx.x % 32 == 0) s_part[threadIdx.x / 32] = dw;
        __syncthreads();
        if (threadIdx.x == 0) {
            float t = 0.0f;
            for (int i = 0; i < 8; ++i) t += s_part[i];
            a.dw[m] = t;
        }
    }
}

}  // namespace

cudaError_t launch_swiglu(int f16, int grad, const SwigluArgs& a, cudaStream_t s) {
    if (f16 && grad) swiglu_kernel<1, 1><<<a.M, 256, 0, s>>>(a);
    else if (f16) swiglu_kernel<1, 0><<<a.M, 256, 0, s>>>(a);
    else if (grad) swiglu_kernel<0, 1><<<a.M, 256, 0, s>>>(a);
    else swiglu_kernel<0, 0><<<a.M, 256, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace moeq
