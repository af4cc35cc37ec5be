// linear.cu - rows times an affine-packed matrix (4 or 8 bits, groups along the input), and the
// matrix itself in bf16 for the products that go over many rows.
//
// Few rows (linear_codes_kernel).  y[t][n] = sum over groups of s * (sum q x) + b * (sum x): the
// codes stay whole numbers inside a group's sum and scale and bias come once per group, so nothing
// but the result is rounded to 16 bits.  The call is bound by the packed bytes (one token: every
// byte is used once), so the work per byte has to stay small: the codes go through warp-level
// tensor-core tiles (mma.sync m16n8k16: 16 matrix rows x 8 tokens), where a nibble becomes the
// bf16 number 128 + q by one and-or of its word, eight codes in seven instructions, and the
// products and sums cost one instruction per 256 codes.  The 128 leaves through the bias:
// s (sum q x) + b (sum x) = s (sum (128 + q) x) + (b - 128 s) (sum x).  An 8-bit code is two
// nibbles, lo + 16 hi, in two accumulators.  (FMAs on the CUDA cores need three instructions per
// code and token; the tcgen05 path needs the matrix unpacked into shared or tensor memory first.)
//
// A dot product does not mind the order of its terms, so a lane takes the k that lie together in
// its words: lane (row r, quarter c) loads a unit's quarter c (a unit is the 64 or 32 inputs that
// one scale covers at least), and the rows of x are staged in shared memory in that order, with the
// sum of each unit beside them.  A block holds 16 matrix rows; its eight warps split the units and
// add their partial sums in shared memory in fixed order.  Blocks stay (two per SM) and walk the
// matrix, each warp's next loads under way while it multiplies: with x staged once per block,
// shared memory and the tensor cores do little, and the loads in flight (16 warps x 4 KB per SM)
// cover the memory's latency.
#include <algorithm>

#include "common.cuh"

namespace moeq {
namespace {

constexpr int kWarps = 8, kThreads = kWarps * 32;
constexpr int kRows = 16;                        // matrix rows of a tile
constexpr int kQuad = 4;                         // units loaded together
constexpr size_t kMaxSmem = 226 * 1024;

__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, "
        "%2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Nibbles j and j + 4 of a word (j = shift / 4) as the bf16 pair {128 + q_j, 128 + q_j+4}.
__device__ __forceinline__ uint32_t nib2(uint32_t w, int shift) { return ((w >> shift) & 0x000F000Fu) | 0x43004300u; }

// Eight bf16 values in the pair order in which the codes leave their words: a 4-bit word gives
// (0, 4) (1, 5) (2, 6) (3, 7); the two 8-bit words give (0, 2) (1, 3), (4, 6) (5, 7).
template <int kBits>
__device__ __forceinline__ uint4 code_order(uint4 u) {
    if (kBits == 4)
        return make_uint4(__byte_perm(u.x, u.z, 0x5410), __byte_perm(u.x, u.z, 0x7632), __byte_perm(u.y, u.w, 0x5410),
                          __byte_perm(u.y, u.w, 0x7632));
    return make_uint4(__byte_perm(u.x, u.y, 0x5410), __byte_perm(u.x, u.y, 0x7632), __byte_perm(u.z, u.w, 0x5410),
                      __byte_perm(u.z, u.w, 0x7632));
}

struct LinArgs {
    moe_qtensor W;
    const uint16_t* x;
    uint16_t* y;
    int T;        // tokens
    int block;    // tokens of a block (<= 8 kNT)
    int units;    // per row
    int vec;      // scales and biases of four units can be loaded together
};

// A quad's words of a tile's 16 rows in a warp's ring, in 16-byte pieces that change places by row so that the
// fragment loads (a unit's quarters of eight rows at once) meet no two in one bank.
template <int kBits, int kUnit>
struct Slot {
    static constexpr int kWords = kUnit * kBits / 128;             // words of a unit's quarter: 1, 2 or 4
    static constexpr int kPieces = kQuad * kWords;                 // 16-byte pieces of a row: 4, 8 or 16
    static constexpr int kCopies = kRows * kPieces / 32;           // per lane
    static constexpr int kBytes = kRows * kPieces * 16 + 2 * kRows * kQuad * 2;  // and the scales and biases
    static constexpr int kDepth = kWords == 4 ? 3 : 4;             // quads in the ring
    __device__ static __forceinline__ int piece(int row, int i) {
        return row * kPieces + (kPieces == 4 ? i ^ (row >> 1 & 3) : kPieces == 8 ? i ^ (row & 7) : i ^ ((row & 1) << 2));
    }
};

__device__ __forceinline__ void cp8(uint32_t dst, const void* src, uint32_t bytes) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp16(uint32_t dst, const void* src, uint32_t bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}

__device__ __forceinline__ float half_of(const uint2& v, int i) {
    const uint32_t w = i / 2 ? v.y : v.x;
    return __uint_as_float(i & 1 ? w & 0xFFFF0000u : w << 16);
}

template <int kBits, int kUnit, int kNT>
__global__ void __launch_bounds__(kThreads, 2) linear_codes_kernel(const LinArgs a) {
    using S = Slot<kBits, kUnit>;
    constexpr int kParts = kUnit / 32;   // 16-byte pieces of x per lane and unit
    extern __shared__ __align__(16) unsigned char sm[];
    const moe_qtensor& W = a.W;
    const int K = W.in, tb = a.block, tb2 = (tb + 1) & ~1, groups = W.in / W.group;
    unsigned char* ring = sm + threadIdx.x / 32 * (S::kDepth * S::kBytes);         // this warp's
    uint4* xs = reinterpret_cast<uint4*>(sm + kWarps * S::kDepth * S::kBytes);     // [unit][part][token][quarter]
    float* xsum = reinterpret_cast<float*>(xs + (size_t)tb * K / 8);               // [unit][tb2]
    float* red = xsum + (size_t)a.units * tb2;                                     // [2][kWarps][kNT * 8][kRows]
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32, g = lane / 4, c = lane % 4;
    const int t0 = blockIdx.y * tb, nt = min(tb, a.T - t0);
    const int tiles = (W.out + kRows - 1) / kRows, quads = (a.units + kQuad - 1) / kQuad;
    const int q0 = (int)((int64_t)quads * warp / kWarps), q1 = (int)((int64_t)quads * (warp + 1) / kWarps);
    const int64_t row_bytes = (int64_t)K * kBits / 8;
    const uint32_t sring = (uint32_t)__cvta_generic_to_shared(ring);

    // copies run kDepth - 1 quads ahead, over the tiles' ends
    int ctile = blockIdx.x, cq = q0, cslot = 0;
    auto copy = [&]() {
        if (ctile < tiles && cq < q1) {
            const uint32_t dst = sring + cslot * S::kBytes;
            const char* src = reinterpret_cast<const char*>(W.packed) + (int64_t)cq * (S::kPieces * 16);
            const int left = (a.units - cq * kQuad) * S::kWords;  // pieces up to the row's end (a unit has kWords)
#pragma unroll
            for (int i = 0; i < S::kCopies; ++i) {
                const int at = i * 32 + lane, row = at / S::kPieces, p = at % S::kPieces;
                const int n = min(ctile * kRows + row, W.out - 1);
                cp16(dst + S::piece(row, p) * 16, src + n * row_bytes + (p < left ? p * 16 : 0), p < left ? 16 : 0);
            }
            if (a.vec) {  // lane: row lane / 2, its scales or its biases
                const int n = min(ctile * kRows + lane / 2, W.out - 1);
                cp8(dst + kRows * S::kPieces * 16 + lane * 8,
                    (lane & 1 ? W.biases : W.scales) + (int64_t)n * groups + cq * kQuad, 8);
            }
            if (++cq == q1) cq = q0, ctile += gridDim.x;
            if (++cslot == S::kDepth) cslot = 0;
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
#pragma unroll
    for (int i = 0; i < S::kDepth - 1; ++i) copy();  // under way while x is staged

    // the block's tokens, in the order of the codes, and the sums of their units
    const int chunks = K / 8;
    for (int i0 = 0; i0 < tb * chunks; i0 += kThreads) {
        const int i = i0 + tid, t = i / chunks, ch = i % chunks;
        uint4 v = make_uint4(0, 0, 0, 0);
        if (t < nt) v = __ldg(reinterpret_cast<const uint4*>(a.x + (int64_t)(t0 + t) * K) + ch);
        float s = 0.0f;
        const uint32_t e[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) s += __uint_as_float(e[j] << 16) + __uint_as_float(e[j] & 0xFFFF0000u);
#pragma unroll
        for (int o = 1; o < kUnit / 8; o <<= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        if (t < tb) {
            const int u = ch / (kUnit / 8), in = ch % (kUnit / 8);
            xs[((int64_t)(u * kParts + in % kParts) * tb + t) * 4 + in / kParts] = code_order<kBits>(v);
            if (in == 0) xsum[u * tb2 + t] = s;
        }
    }
    if (tb < tb2)
        for (int u = tid; u < a.units; u += kThreads) xsum[u * tb2 + tb] = 0.0f;
    __syncthreads();

    int slot = 0;
    for (int tile = blockIdx.x, buf = 0; tile < tiles; tile += gridDim.x, buf ^= 1) {
        float y[kNT][4];
#pragma unroll
        for (int n = 0; n < kNT; ++n)
#pragma unroll
            for (int j = 0; j < 4; ++j) y[n][j] = 0.0f;
        for (int qi = q0; qi < q1; ++qi) {
            uint2 sc[2], bi[2];  // scales and biases of the quad, bf16 pairs
            if (!a.vec) {
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const int64_t at = (int64_t)min(tile * kRows + g + 8 * r, W.out - 1) * groups;
                    uint32_t e[2][kQuad];
#pragma unroll
                    for (int i = 0; i < kQuad; ++i) {
                        const int gi = min(qi * kQuad + i, a.units - 1) * kUnit / W.group;
                        e[0][i] = __ldg(W.scales + at + gi);
                        e[1][i] = __ldg(W.biases + at + gi);
                    }
                    sc[r] = make_uint2(e[0][0] | e[0][1] << 16, e[0][2] | e[0][3] << 16);
                    bi[r] = make_uint2(e[1][0] | e[1][1] << 16, e[1][2] | e[1][3] << 16);
                }
            }
            asm volatile("cp.async.wait_group %0;" ::"n"(S::kDepth - 2) : "memory");
            __syncwarp();
            copy();  // into the slot of the quad before this one
            const unsigned char* q = ring + slot * S::kBytes;
            if (++slot == S::kDepth) slot = 0;
            if (a.vec) {
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const uint4 v = *reinterpret_cast<const uint4*>(q + kRows * S::kPieces * 16 + (g + 8 * r) * 16);
                    sc[r] = make_uint2(v.x, v.y);
                    bi[r] = make_uint2(v.z, v.w);
                }
            }
#pragma unroll
            for (int i = 0; i < kQuad; ++i) {
                const int u = qi * kQuad + i;
                if (u >= a.units) break;
                uint32_t w[2][S::kWords];
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const unsigned char* pw = q + S::piece(g + 8 * r, i * S::kWords + c * S::kWords / 4) * 16;
                    if constexpr (S::kWords == 4) {
                        const uint4 v = *reinterpret_cast<const uint4*>(pw);
                        w[r][0] = v.x, w[r][1] = v.y, w[r][2] = v.z, w[r][3] = v.w;
                    } else if constexpr (S::kWords == 2) {
                        const uint2 v = *reinterpret_cast<const uint2*>(pw + c % 2 * 8);
                        w[r][0] = v.x, w[r][1] = v.y;
                    } else {
                        w[r][0] = *reinterpret_cast<const uint32_t*>(pw + c * 4);
                    }
                }
                const float s0 = half_of(sc[0], i), s1 = half_of(sc[1], i);
                constexpr float kOff = kBits == 4 ? 128.0f : 128.0f * 17.0f;
                const float b0 = fmaf(-kOff, s0, half_of(bi[0], i)), b1 = fmaf(-kOff, s1, half_of(bi[1], i));
#pragma unroll
                for (int n = 0; n < kNT; ++n) {
                    float lo[4] = {0, 0, 0, 0}, hi[4] = {0, 0, 0, 0};
#pragma unroll
                    for (int p = 0; p < kParts; ++p) {
                        uint4 x = make_uint4(0, 0, 0, 0);
                        if (8 * n + g < tb) x = xs[((int64_t)(u * kParts + p) * tb + 8 * n + g) * 4 + c];
                        if constexpr (kBits == 4) {  // one word: eight codes
                            const uint32_t w0 = w[0][p], w1 = w[1][p];
                            mma16816(lo, nib2(w0, 0), nib2(w1, 0), nib2(w0, 4), nib2(w1, 4), x.x, x.y);
                            mma16816(lo, nib2(w0, 8), nib2(w1, 8), nib2(w0, 12), nib2(w1, 12), x.z, x.w);
                        } else {                     // two words: eight codes, low and high nibbles
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                const uint32_t w0 = w[0][2 * p + h], w1 = w[1][2 * p + h];
                                const uint32_t x0 = h ? x.z : x.x, x1 = h ? x.w : x.y;
                                mma16816(lo, nib2(w0, 0), nib2(w1, 0), nib2(w0, 8), nib2(w1, 8), x0, x1);
                                mma16816(hi, nib2(w0, 4), nib2(w1, 4), nib2(w0, 12), nib2(w1, 12), x0, x1);
                            }
                        }
                    }
                    float2 xt = make_float2(0.0f, 0.0f);
                    if (8 * n + 2 * c < tb) xt = *reinterpret_cast<const float2*>(&xsum[u * tb2 + 8 * n + 2 * c]);
                    if constexpr (kBits == 8) {
#pragma unroll
                        for (int j = 0; j < 4; ++j) lo[j] = fmaf(16.0f, hi[j], lo[j]);
                    }
                    y[n][0] += fmaf(s0, lo[0], b0 * xt.x);
                    y[n][1] += fmaf(s0, lo[1], b0 * xt.y);
                    y[n][2] += fmaf(s1, lo[2], b1 * xt.x);
                    y[n][3] += fmaf(s1, lo[3], b1 * xt.y);
                }
            }
        }
        // the warps' parts, added in fixed order
        float* rb = red + buf * (kWarps * kNT * 8 * kRows);
#pragma unroll
        for (int n = 0; n < kNT; ++n)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                rb[(warp * kNT * 8 + 8 * n + 2 * c + j % 2) * kRows + g + 8 * (j / 2)] = y[n][j];
        __syncthreads();
        for (int i = tid; i < nt * kRows; i += kThreads) {
            float v = 0.0f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) v += rb[w * kNT * 8 * kRows + i];
            const int n = tile * kRows + i % kRows;
            if (n < W.out) a.y[(int64_t)(t0 + i / kRows) * W.out + n] = f2bf16(v);
        }
    }
}

// The matrix in bf16: eight codes (one 4-bit word or two 8-bit ones) to one 16-byte store a thread; bound by
// the 2 bytes written per weight.  One rounding per weight (s q + b in fp32 is exact to its last place): the
// tensor core multiplies 16-bit operands, and the rows it meets are rounded to as many bits.
template <int kBits>
__global__ void __launch_bounds__(256) dequant16_kernel(const moe_qtensor W, int64_t pieces, uint4* __restrict__ out) {
    const int groups8 = W.group / 8;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < pieces; i += (int64_t)gridDim.x * 256) {
        uint32_t w[2];
        if (kBits == 4) {
            w[0] = __ldg(W.packed + i);
            w[1] = w[0] >> 16;
        } else {
            const uint2 v = __ldg(reinterpret_cast<const uint2*>(W.packed) + i);
            w[0] = v.x;
            w[1] = v.y;
        }
        const int64_t g = i / groups8;  // (a row is a whole number of groups)
        const float s = bf16f(__ldg(W.scales + g)), b = bf16f(__ldg(W.biases + g));
        uint32_t o[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t v = w[j / 2] >> (2 * kBits * (j % 2));
            const float lo = fmaf(s, u2f_small(v & ((1u << kBits) - 1u)), b);
            const float hi = fmaf(s, u2f_small((v >> kBits) & ((1u << kBits) - 1u)), b);
            o[j] = (uint32_t)f2bf16(lo) | ((uint32_t)f2bf16(hi) << 16);
        }
        out[i] = make_uint4(o[0], o[1], o[2], o[3]);
    }
}

int sm_count() {
    int dev = 0, n = 148;
    cudaGetDevice(&dev);
    cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
    return n;
}

template <int kBits, int kUnit>
size_t codes_smem(const moe_qtensor& W, int tb) {
    using S = Slot<kBits, kUnit>;
    return (size_t)kWarps * S::kDepth * S::kBytes + (size_t)tb * W.in * 2 +
           (size_t)(W.in / kUnit) * ((tb + 1) & ~1) * 4 + 2u * kWarps * (tb > 8 ? 16 : 8) * kRows * sizeof(float);
}

template <int kBits, int kUnit, int kNT>
cudaError_t launch_codes(LinArgs a, cudaStream_t s) {
    const size_t smem = codes_smem<kBits, kUnit>(a.W, a.block);
    const cudaError_t e = cudaFuncSetAttribute((const void*)linear_codes_kernel<kBits, kUnit, kNT>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    const int tiles = (a.W.out + kRows - 1) / kRows, across = (a.T + a.block - 1) / a.block;
    const int room = std::max(1, (smem > 113 * 1024 ? 1 : 2) * sm_count() / across);
    linear_codes_kernel<kBits, kUnit, kNT><<<dim3(std::min(tiles, room), across), kThreads, smem, s>>>(a);
    return cudaGetLastError();
}

template <int kBits, int kUnit>
cudaError_t launch_unit(LinArgs a, cudaStream_t s) {
    a.units = a.W.in / kUnit;
    a.vec = a.W.group == kUnit && a.units % kQuad == 0 && ((uintptr_t)a.W.scales & 7) == 0 &&
            ((uintptr_t)a.W.biases & 7) == 0;
    // as many tokens a block as one or two token tiles hold and shared memory takes
    int tb = std::min(a.T, 16);
    while (tb > 1 && codes_smem<kBits, kUnit>(a.W, tb) > kMaxSmem) --tb;
    const int blocks = (a.T + tb - 1) / tb;
    a.block = (a.T + blocks - 1) / blocks;
    return a.block > 8 ? launch_codes<kBits, kUnit, 2>(a, s) : launch_codes<kBits, kUnit, 1>(a, s);
}

}  // namespace

// Whether a row of x, and the ring beside it, fit in shared memory (from about 54,000 8-bit inputs on they do not).
bool affine_codes_supported(const moe_qtensor& W) {
    const size_t smem = W.group % 64 == 0 ? (W.bits == 4 ? codes_smem<4, 64>(W, 1) : codes_smem<8, 64>(W, 1))
                                          : (W.bits == 4 ? codes_smem<4, 32>(W, 1) : codes_smem<8, 32>(W, 1));
    return smem <= kMaxSmem;
}

cudaError_t launch_affine_linear(const moe_qtensor& W, const uint16_t* x, int T, uint16_t* y, cudaStream_t s) {
    LinArgs a;
    a.W = W;
    a.x = x;
    a.y = y;
    a.T = T;
    if (W.group % 64 == 0) return W.bits == 4 ? launch_unit<4, 64>(a, s) : launch_unit<8, 64>(a, s);
    return W.bits == 4 ? launch_unit<4, 32>(a, s) : launch_unit<8, 32>(a, s);
}

cudaError_t launch_affine_dequant16(const moe_qtensor& W, uint16_t* out, cudaStream_t s) {
    const int64_t pieces = (int64_t)W.out * W.in / 8, want = (pieces + 255) / 256;
    const unsigned blocks = (unsigned)std::min<int64_t>(want, (int64_t)sm_count() * 8);
    if (W.bits == 4) dequant16_kernel<4><<<blocks, 256, 0, s>>>(W, pieces, reinterpret_cast<uint4*>(out));
    else dequant16_kernel<8><<<blocks, 256, 0, s>>>(W, pieces, reinterpret_cast<uint4*>(out));
    return cudaGetLastError();
}

}  // namespace moeq
