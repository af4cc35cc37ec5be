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
// (begin >= end: no rows)
__device__ __forceinline__ Range rows_of(const SwigluArgs& a) {
    if (!a.off) return Range{0, a.M};
    return Range{max(ld_after(a.off), 0), min(ld_after(a.off + a.G), a.M)};
}

// sigmoid(g) without overflow: e = exp(-|g|) <= 1 and 1 + e in [1, 2].  As a power of two, whose argument is rounded:
// e is off by 1.5 |g| 2^-24 of itself, a loss only where e is already small (forward at 16384 x 512: 11.0
// us, with expf 12.6, with no exponential at all 10.2).
__device__ __forceinline__ float sigmoid(float g) {
    const float e = exp2f(-1.4426950408889634f * fabsf(g)), r = __fdividef(1.0f, 1.0f + e);
    return g >= 0.0f ? r : e * r;
}

struct Elem {  // what one element contributes
    float h, dg, du, dw;
};
template <int kGrad>
__device__ __forceinline__ Elem element(float g, float u, float w, float d) {
    const float s = sigmoid(g), sl = g * s;
    Elem e;
    if (!kGrad) {
        e.h = w * sl * u;
    } else {
        const float wd = w * d;
        e.dg = wd * u * s * (1.0f + g * (1.0f - s));
        e.du = wd * sl;
        e.dw = d * (sl * u);
    }
    return e;
}

__device__ __forceinline__ float lane16(const uint4& v, int i, int f16) {
    const uint32_t w = i / 2 == 0 ? v.x : i / 2 == 1 ? v.y : i / 2 == 2 ? v.z : v.w;
    const uint16_t h = (uint16_t)(i % 2 ? w >> 16 : w & 0xFFFFu);
    return f16 ? ld16<1>(h) : ld16<0>(h);
}
template <int kF16>
__device__ __forceinline__ uint4 pack8(const float (&v)[8]) {
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = (uint32_t)st16<kF16>(v[2 * i]) | ((uint32_t)st16<kF16>(v[2 * i + 1]) << 16);
    return make_uint4(o[0], o[1], o[2], o[3]);
}

// Rows of whole 16-byte pieces: kTeam threads a row (a warp, or a block for wide rows), eight elements a thread and
// step.  Bound by memory: 6 bytes an element forward, 10 for the gradient; a thread's loads of a step go out together
// and a few thousand rows keep every SM's warps full (16380 x 512 forward 10.6 us, 4.7 TB/s; 15360 x 1024 gradient 28
// us, 5.6 TB/s).
template <int kF16, int kGrad, int kTeam>
__global__ void __launch_bounds__(256) swiglu_vec_kernel(const SwigluArgs a) {
    __shared__ float s_part[8];
    grid_wait();
    const Range r = rows_of(a);
    const int I8 = a.I / 8, at = threadIdx.x % kTeam;
    for (int64_t m = r.begin + (int64_t)blockIdx.x * (256 / kTeam) + threadIdx.x / kTeam; m < r.end;
         m += (int64_t)gridDim.x * (256 / kTeam)) {
        const uint4 *gr = reinterpret_cast<const uint4*>(a.gu + m * 2 * a.I), *ur = gr + I8;
        const uint4* dr = reinterpret_cast<const uint4*>(a.dh + m * a.I);
        const float w = a.w ? ld_after(a.w + m) : 1.0f;
        float dw = 0.0f;
#pragma unroll 2
        for (int i = at; i < I8; i += kTeam) {
            const uint4 g = ld_after_once(gr + i), u = ld_after_once(ur + i);
            uint4 d = make_uint4(0, 0, 0, 0);
            if (kGrad) d = ld_after_once(dr + i);
            float o1[8], o2[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const Elem e = element<kGrad>(lane16(g, j, kF16), lane16(u, j, kF16), w, lane16(d, j, kF16));
                o1[j] = kGrad ? e.dg : e.h;
                o2[j] = kGrad ? e.du : 0.0f;
                if (kGrad) dw += e.dw;
            }
            if (kGrad) {
                uint4* o = reinterpret_cast<uint4*>(a.dgu + m * 2 * a.I);
                o[i] = pack8<kF16>(o1);
                o[I8 + i] = pack8<kF16>(o2);
            } else {
                reinterpret_cast<uint4*>(a.h + m * a.I)[i] = pack8<kF16>(o1);
            }
        }
        if (kGrad && a.dw) {
            dw = warp_sum(dw);
            if (kTeam == 32) {
                if (at == 0) a.dw[m] = dw;
            } else {
                if (threadIdx.x % 32 == 0) s_part[threadIdx.x / 32] = dw;
                __syncthreads();
                if (threadIdx.x == 0) {
                    float t = 0.0f;
                    for (int i = 0; i < 8; ++i) t += s_part[i];
                    a.dw[m] = t;
                }
                __syncthreads();
            }
        }
    }
}

// Any size and alignment: one block per row, the loads of kAhead elements a thread under way together (16384 rows of 1001
// 26.8 us, gradient 43.3; one by one, behind the ordered loads, 41.8 and 62.7).
constexpr int kAhead = 4;
template <int kF16, int kGrad>
__global__ void __launch_bounds__(256) swiglu_any_kernel(const SwigluArgs a) {
    __shared__ float s_part[8];
    grid_wait();
    const Range r = rows_of(a);
    const int64_t m = blockIdx.x;
    if (m < r.begin || m >= r.end) return;
    const int I = a.I;
    const uint16_t *gr = a.gu + m * 2 * I, *ur = gr + I, *dr = a.dh + m * I;
    const float w = a.w ? ld_after(a.w + m) : 1.0f;
    float dw = 0.0f;
    for (int i0 = threadIdx.x; i0 < I; i0 += 256 * kAhead) {
        uint16_t g[kAhead], u[kAhead], d[kAhead];
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            const int i = i0 + 256 * j;
            if (i >= I) continue;
            g[j] = ld_after(gr + i);
            u[j] = ld_after(ur + i);
            if (kGrad) d[j] = ld_after(dr + i);
        }
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            const int i = i0 + 256 * j;
            if (i >= I) continue;
            const Elem e = element<kGrad>(ld16<kF16>(g[j]), ld16<kF16>(u[j]), w, kGrad ? ld16<kF16>(d[j]) : 0.0f);
            if (!kGrad) {
                a.h[m * I + i] = st16<kF16>(e.h);
            } else {
                a.dgu[m * 2 * I + i] = st16<kF16>(e.dg);
                a.dgu[m * 2 * I + I + i] = st16<kF16>(e.du);
                dw += e.dw;
            }
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

constexpr int kWide = 4096;  // from this width on a block takes a row

template <int kF16, int kGrad>
cudaError_t launch_typed(const SwigluArgs& a, cudaStream_t s) {
    const uintptr_t all = (uintptr_t)a.gu | (uintptr_t)(kGrad ? (const void*)a.dh : a.h) | (kGrad ? (uintptr_t)a.dgu : 0);
    if (a.I % 8 || (all & 15)) {
        return launch_dependent(swiglu_any_kernel<kF16, kGrad>, dim3(a.M), 256, 0, 1, s, a);
    }
    if (a.I >= kWide) return launch_dependent(swiglu_vec_kernel<kF16, kGrad, 256>, dim3(a.M), 256, 0, 1, s, a);
    return launch_dependent(swiglu_vec_kernel<kF16, kGrad, 32>, dim3((a.M + 7) / 8), 256, 0, 1, s, a);
}

}  // namespace

cudaError_t launch_swiglu(int f16, int grad, const SwigluArgs& a, cudaStream_t s) {
    if (f16) return grad ? launch_typed<1, 1>(a, s) : launch_typed<1, 0>(a, s);
    return grad ? launch_typed<0, 1>(a, s) : launch_typed<0, 0>(a, s);
}

}  // namespace moeq
