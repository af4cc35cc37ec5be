// linear.cu - rows times an affine-packed matrix (4 or 8 bits, groups along the input), and the
// matrix itself in bf16 for the products that go over many rows.
//
// Few rows (linear_codes_kernel).  y[t][n] = sum over groups of s * (sum q x) + b * (sum x): the
// codes stay whole numbers inside a group's sum and scale and bias come once per group, so nothing
// but the result is rounded to 16 bits.  The call is bound by the packed bytes (one token: every
// byte is used once), so the work per byte has to stay small: the codes go through warp-level
// tensor-core tiles (mma.sync m16n8k16: 16 matrix rows x 8 tokens), where a code masked out of its
// word is a number already: the fp16 subnormal q 2^-24, or 16 q 2^-24 where it lies four bits higher
// (x is divided by 16 there).  Eight 4-bit codes take five instructions, four 8-bit ones three, and
// the products and sums one per 256 codes.  x enters as fp16 too, scaled by a power of two per unit
// (the 64 or 32 inputs that one scale covers at least), so that the unit's largest magnitude lies in
// [2^14, 2^15): bf16 values down to 2^-27 of that are exact, smaller ones off by 2^-35 of it at most.
// (With nibbles as bf16 numbers 128 + q, an or more each, and bytes in two halves: one token to 131072
// outputs 36.1 us against 34.1 at the time, 8-bit 4096 to 16384 21.3 against 18.4.  As e4m3 numbers, with x in two
// e4m3 parts, 38.1: these products are conversions and 16-bit ones on this GPU.  FMAs on the CUDA
// cores need three instructions per code and token; the tcgen05 path needs the matrix unpacked first.)
//
// A dot product does not mind the order of its terms, so a lane takes the k that lie together in its
// words: lane (row r, quarter c) loads a unit's quarter c, and the rows of x are staged in shared
// memory in that order, with the sum and the scale of each unit beside them.  Tall matrices give
// every warp tiles of its own; where there are too few tiles, two, four or eight warps of a block
// split a tile's units and add their partial sums in shared memory in fixed order.  Blocks stay (two
// per SM) and walk the matrix, each warp with a ring of its own that asynchronous copies fill one to
// three quads (four units of a tile) ahead: x is staged once per block, and the copies in flight
// cover the memory's latency.
//
// What bounds it.  Small matrices: the launch and one pass through memory (2048 x 512, one token: 3.1
// us).  Tall ones (2048 to 131072, one token: 33.1 us, 4.6 TB/s of the packed bytes; with loads to registers
// and every tile added up by eight warps 57): no unit is full.  Of the active cycles the path to shared memory is busy in
// 69 %, the issue slots in 56, the integer pipe in 49, the tensor pipe in 24, DRAM in 51 of all; 14.5 warps a
// multiprocessor, of whose 6.5 cycles an instruction 1.2 are its own latency, 1.1 another warp's turn, 0.8 shared memory,
// 0.8 a busy pipe, 0.5 each barriers and loads from memory.
//
// Many rows.  dequant16_kernel writes the matrix out in bf16 and the tcgen05 kernel of the grouped
// products multiplies it (2048 tokens, 2048 to 4096: 32 us, 6 of them for the copy).  Unpacking inside
// that kernel, by 8 or 16 warps that fill its stages, took 38 to 47: a stage's 8192 codes cost those
// warps more than its products cost the tensor core.
#include <cuda_fp16.h>

#include <algorithm>

#include "common.cuh"

namespace moeq {
namespace {

constexpr int kWarps = 8, kThreads = kWarps * 32;
constexpr int kQuad = 4;                         // units loaded together
constexpr size_t kMaxSmem = 226 * 1024;

__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, "
        "%2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// The same from zero.
__device__ __forceinline__ void mma16816_0(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                           uint32_t b1) {
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, "
        "%10, %10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}

// The codes of a word as the fp16 numbers whose bits they are, the subnormals q 2^-24: pairs (0, 4) (1, 5) (2, 6) (3, 7)
// of a 4-bit word, the second and fourth 16 times as large, or (0, 2) (1, 3) of an 8-bit one.
template <int kBits>
__device__ __forceinline__ uint32_t codes2(uint32_t w, int j) {
    if (kBits == 8) return (j ? w >> 8 : w) & 0x00FF00FFu;
    return (j & 2 ? w >> 8 : w) & (j & 1 ? 0x00F000F0u : 0x000F000Fu);
}

__device__ __forceinline__ uint32_t half_pair(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}

// Eight bf16 values times `scale` as fp16 in the pair order in which the codes leave their words, a sixteenth of them
// where the codes are 16 times as large.
template <int kBits>
__device__ __forceinline__ uint4 code_order(const uint4& u, float scale) {
    const uint32_t e[4] = {u.x, u.y, u.z, u.w};
    float x[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        x[2 * j] = __uint_as_float(e[j] << 16) * scale;
        x[2 * j + 1] = __uint_as_float(e[j] & 0xFFFF0000u) * scale;
    }
    if (kBits == 8)
        return make_uint4(half_pair(x[0], x[2]), half_pair(x[1], x[3]), half_pair(x[4], x[6]), half_pair(x[5], x[7]));
    constexpr float k16 = 0.0625f;
    return make_uint4(half_pair(x[0], x[4]), half_pair(x[1] * k16, x[5] * k16), half_pair(x[2], x[6]),
                      half_pair(x[3] * k16, x[7] * k16));
}

struct LinArgs {
    moe_qtensor W;
    const uint16_t* x;
    uint16_t* y;
    int T;        // tokens
    int block;    // tokens of a block (<= 8 kNT)
    int units;    // per row
    int split;    // warps that share a tile: 1, 2, 4 or 8
    uint32_t inv_span;  // ceil(2^32 / units of a group), 0 for one
    // of a row's 16-byte pieces: ceil(2^32 / pieces), and how far kThreads of them lead (rows, pieces)
    uint32_t inv_chunks;
    int step_t, step_c;
};

// A quad's words of a tile's rows in a warp's ring, in 16-byte pieces that change places by row so that the
// fragment loads (a unit's quarters of eight rows at once) meet no two in one bank.
template <int kBits, int kUnit, int kMT>
struct Slot {
    static constexpr int kRows = 16 * kMT;                         // matrix rows of a tile
    static constexpr int kWords = kUnit * kBits / 128;             // words of a unit's quarter: 1, 2 or 4
    static constexpr int kPieces = kQuad * kWords;                 // 16-byte pieces of a row: 4, 8 or 16
    static constexpr int kCopies = kRows * kPieces / 32;           // per lane
    static constexpr int kBytes = kRows * kPieces * 16 + 2 * kRows * kQuad * 2;  // and the scales and biases
    static constexpr int kDepth = kMT == 2 ? 2 : kWords == 4 ? 3 : 4;            // quads in the ring
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

__device__ __forceinline__ uint4 lds128(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
    return v;
}
__device__ __forceinline__ void sts64(uint32_t a, uint32_t x, uint32_t y) {
    asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(a), "r"(x), "r"(y) : "memory");
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
    return v;
}
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
    uint32_t v;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a));
    return v;
}

__device__ __forceinline__ float half_of(const uint2& v, int i) {
    const uint32_t w = i / 2 ? v.y : v.x;
    return __uint_as_float(i & 1 ? w & 0xFFFF0000u : w << 16);
}

// A unit's x is scaled by 2^(14 - e) for the exponent e of its largest magnitude; its product with codes q 2^-24 is
// scaled back by 2^e, and the 2^10 that is left once at the end.
constexpr float kBack = 0x1p10f;
constexpr int kAhead = 4;  // pieces of x a thread has under way

// kVec: the scales and biases of four units can be copied together.
template <int kBits, int kUnit, int kNT, int kMT, int kVec>
__global__ void __launch_bounds__(kThreads, 2) linear_codes_kernel(const LinArgs a) {
    using S = Slot<kBits, kUnit, kMT>;
    constexpr int kParts = kUnit / 32;   // 16-byte pieces of x per lane and unit
    constexpr int kRows = S::kRows, kRed = kNT * 8 * kRows;
    extern __shared__ __align__(16) unsigned char sm[];
    const moe_qtensor& W = a.W;
    const int K = W.in, tb = a.block, tb2 = (tb + 1) & ~1, groups = W.in / W.group;
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32, g = lane / 4, c = lane % 4;
    unsigned char* ring = sm + warp * (S::kDepth * S::kBytes);                     // this warp's
    // x: [unit][token][quarter and part], a unit's 16-byte pieces of two neighbouring tokens in opposite halves (else
    // they would share banks); then a block of zeros that the lanes of tokens past the last read
    uint4* xs = reinterpret_cast<uint4*>(sm + kWarps * S::kDepth * S::kBytes);
    const int xunit = tb * 4 * kParts;                                             // pieces of a unit
    uint4* zeros = xs + (size_t)a.units * xunit;
    float* xsum = reinterpret_cast<float*>(zeros + 4 * kParts);                    // [unit][two tokens]{sums, 2^e}, then zeros
    float* red = xsum + (size_t)a.units * tb2 * 2 + 4;                             // [2][kWarps][kRed]
    const int t0 = blockIdx.y * tb, nt = min(tb, a.T - t0);
    const int tiles = (W.out + kRows - 1) / kRows, quads = (a.units + kQuad - 1) / kQuad;
    // the block's warps: kWarps / split tiles at a time, `split` of them to a tile's units
    const int split = a.split, part = warp % split, across = kWarps / split;
    const int q0 = (int)((int64_t)quads * part / split), q1 = (int)((int64_t)quads * (part + 1) / split);
    const int first = blockIdx.x * across + warp / split, stride = gridDim.x * across;
    const int row_bytes = K * kBits / 8;
    const uint32_t sring = (uint32_t)__cvta_generic_to_shared(ring);

    // copies run kDepth - 1 quads ahead, over the tiles' ends; a lane's pieces are kStep rows apart
    constexpr int kStep = 32 / S::kPieces;
    const int crow = lane / S::kPieces, cp = lane % S::kPieces;
    int ctile = first, cq = q0, cslot = 0;
    // Scales and biases that no aligned copy fetches are loaded one quad's work before they are stored beside the codes
    // (loaded where they are used instead: 2880 inputs to 19168, one token 17.3 us against 14.3).
    uint32_t pend[kMT][kQuad];
    int pslot = -1;
    auto copy = [&]() {
        if (!kVec && pslot >= 0) {
            const uint32_t dst = sring + pslot * S::kBytes + kRows * S::kPieces * 16 + lane * 8;
#pragma unroll
            for (int m = 0; m < kMT; ++m)
                sts64(dst + m * 256, pend[m][0] | pend[m][1] << 16, pend[m][2] | pend[m][3] << 16);
            pslot = -1;
        }
        if (ctile < tiles && cq < q1) {
            const uint32_t dst = sring + cslot * S::kBytes;
            const char* src = reinterpret_cast<const char*>(W.packed) + (int64_t)ctile * kRows * row_bytes +
                              cq * (S::kPieces * 16);
            const int left = (a.units - cq * kQuad) * S::kWords;  // pieces up to the row's end (a unit has kWords)
            const int last = W.out - 1 - ctile * kRows;            // the tile's last row
            if (left >= S::kPieces && last >= kRows - 1) {
                const char* p = src + crow * row_bytes + cp * 16;
#pragma unroll
                for (int i = 0; i < S::kCopies; ++i, p += kStep * row_bytes)
                    cp16(dst + S::piece(i * kStep + crow, cp) * 16, p, 16);
            } else {
#pragma unroll
                for (int i = 0; i < S::kCopies; ++i)
                    cp16(dst + S::piece(i * kStep + crow, cp) * 16,
                         src + min(i * kStep + crow, last) * row_bytes + (cp < left ? cp * 16 : 0), cp < left ? 16 : 0);
            }
            // lane: row lane / 2 (and 16 further), its scales or its biases
            const uint16_t* sb = (lane & 1 ? W.biases : W.scales) + (int64_t)ctile * kRows * groups;
            if (kVec) {
                sb += cq * kQuad;
#pragma unroll
                for (int m = 0; m < kMT; ++m)
                    cp8(dst + kRows * S::kPieces * 16 + (m * 32 + lane) * 8, sb + min(m * 16 + lane / 2, last) * groups, 8);
            }
            if (!kVec) {
                pslot = cslot;
#pragma unroll
                for (int i = 0; i < kQuad; ++i) {
                    const uint32_t u = min(cq * kQuad + i, a.units - 1), gi = a.inv_span ? __umulhi(u, a.inv_span) : u;
#pragma unroll
                    for (int m = 0; m < kMT; ++m)
                        pend[m][i] = ld_after(sb + (int64_t)min(m * 16 + lane / 2, last) * groups + gi);
                }
            }
            if (++cq == q1) cq = q0, ctile += stride;
            if (++cslot == S::kDepth) cslot = 0;
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    grid_wait();
#pragma unroll
    for (int i = 0; i < S::kDepth - 1; ++i) copy();  // under way while x is staged

    // the block's tokens, in the order of the codes, with the scales and the sums of their units
    const int chunks = K / 8;
    int t = (int)__umulhi(tid, a.inv_chunks), ch = tid - t * chunks;
    for (int i0 = 0; i0 < tb * chunks; i0 += kAhead * kThreads) {
        uint4 v[kAhead];
        int tt[kAhead], cc[kAhead];
#pragma unroll
        for (int h = 0; h < kAhead; ++h) {
            tt[h] = t, cc[h] = ch;
            v[h] = make_uint4(0, 0, 0, 0);
            if (t < nt) v[h] = ld_after(reinterpret_cast<const uint4*>(a.x + (int64_t)(t0 + t) * K) + ch);
            t += a.step_t, ch += a.step_c;
            if (ch >= chunks) ch -= chunks, ++t;
        }
#pragma unroll
        for (int h = 0; h < kAhead; ++h) {
            if (i0 + h * kThreads >= tb * chunks) break;
            float s = 0.0f;
            const uint32_t e[4] = {v[h].x, v[h].y, v[h].z, v[h].w};
            constexpr uint32_t k = 0x7FFF7FFFu;  // magnitudes
            uint32_t top = __vmaxu2(__vmaxu2(e[0] & k, e[1] & k), __vmaxu2(e[2] & k, e[3] & k));
#pragma unroll
            for (int j = 0; j < 4; ++j) s += __uint_as_float(e[j] << 16) + __uint_as_float(e[j] & 0xFFFF0000u);
#pragma unroll
            for (int o = 1; o < kUnit / 8; o <<= 1) {
                s += __shfl_xor_sync(0xffffffffu, s, o);
                top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, o));
            }
            if (tt[h] < tb) {
                const int u = cc[h] / (kUnit / 8), in = cc[h] % (kUnit / 8), to = tt[h];
                // 2^(14 - (E - 127)) for the exponent field E of the unit's largest magnitude (16 at least), which
                // brings that to [2^14, 2^15)
                const uint32_t E = max(max(top & 0xFFFFu, top >> 16) >> 7, 16u);
                xs[u * xunit + to * 4 * kParts + ((in % kParts) ^ (kParts == 2 ? to & 1 : 0)) * 4 + in / kParts] =
                    code_order<kBits>(v[h], __uint_as_float((268u - E) << 23));
                if (in == 0) {  // (an infinity or NaN is in the sum)
                    float* f = xsum + (u * tb2 + (to & ~1)) * 2 + (to & 1);
                    f[0] = s / kBack;
                    f[2] = __uint_as_float(min(E, 254u) << 23);
                }
            }
        }
    }
    if (tb < tb2)
        for (int u = tid; u < a.units; u += kThreads)
            xsum[(u * tb2 + tb - 1) * 2 + 1] = xsum[(u * tb2 + tb - 1) * 2 + 3] = 0.0f;
    if (tid < 4 * kParts) zeros[tid] = make_uint4(0, 0, 0, 0);
    if (tid < 4) xsum[a.units * tb2 * 2 + tid] = 0.0f;
    __syncthreads();
    // where this lane's pieces of x and sums start, and how far apart its units are (shared memory addresses: the
    // integer pipe that unpacks the codes has no room for address arithmetic)
    uint32_t xp[kNT][kParts], sp[kNT], xstep[kNT], sstep[kNT];
#pragma unroll
    for (int n = 0; n < kNT; ++n) {
        const int t = 8 * n + g;
        xstep[n] = t < tb ? xunit * 16 : 0;
#pragma unroll
        for (int p = 0; p < kParts; ++p)
            xp[n][p] = (uint32_t)__cvta_generic_to_shared(t < tb ? xs + t * 4 * kParts : zeros) +
                       ((p ^ (kParts == 2 ? t & 1 : 0)) * 4 + c) * 16;
        const bool in = 8 * n + 2 * c < tb;
        sstep[n] = in ? tb2 * 8 : 0;
        sp[n] = (uint32_t)__cvta_generic_to_shared(xsum + (in ? 8 * n + 2 * c : a.units * tb2) * 2);
    }
    uint32_t wp[kQuad];  // and its quarter of a unit's words within a slot, for the first of its rows
#pragma unroll
    for (int i = 0; i < kQuad; ++i)
        wp[i] = S::piece(g, i * S::kWords + c * S::kWords / 4) * 16 + (S::kWords == 4 ? 0 : S::kWords == 2 ? c % 2 * 8 : c * 4);
    const uint32_t cp_s = kRows * S::kPieces * 16 + g * 16;

    int slot = 0;
    // (warps that share tiles go as many rounds as the block's first one)
    for (int tile = first, buf = 0; (split == 1 ? tile : tile - warp / split) < tiles; tile += stride, buf ^= 1) {
        float y[kMT][kNT][4];
#pragma unroll
        for (int m = 0; m < kMT; ++m)
#pragma unroll
            for (int n = 0; n < kNT; ++n)
#pragma unroll
                for (int j = 0; j < 4; ++j) y[m][n][j] = 0.0f;
        for (int qi = q0; qi < q1 && tile < tiles; ++qi) {
            uint2 sc[kMT][2], bi[kMT][2];  // scales and biases of the quad, bf16 pairs
            asm volatile("cp.async.wait_group %0;" ::"n"(S::kDepth - 2) : "memory");
            __syncwarp();
            copy();  // into the slot of the quad before this one
            const uint32_t q = sring + slot * S::kBytes;
            if (++slot == S::kDepth) slot = 0;
            if (!kVec) __syncwarp();
#pragma unroll
            for (int r = 0; r < 2 * kMT; ++r) {
                const uint4 v = lds128(q + cp_s + 8 * r * 16);
                sc[r / 2][r % 2] = make_uint2(v.x, v.y);
                bi[r / 2][r % 2] = make_uint2(v.z, v.w);
            }
#pragma unroll
            for (int i = 0; i < kQuad; ++i) {
                const int u = qi * kQuad + i;
                if (u >= a.units) break;
                uint4 x[kNT][kParts];
                float4 xt[kNT];
#pragma unroll
                for (int n = 0; n < kNT; ++n) {
#pragma unroll
                    for (int p = 0; p < kParts; ++p) x[n][p] = lds128(xp[n][p] + u * xstep[n]);
                    const uint4 v = lds128(sp[n] + u * sstep[n]);
                    xt[n] = make_float4(__uint_as_float(v.x), __uint_as_float(v.y), __uint_as_float(v.z), __uint_as_float(v.w));
                }
#pragma unroll
                for (int m = 0; m < kMT; ++m) {
                    uint32_t w[2][S::kWords];
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        const uint32_t pw = q + wp[i] + (16 * m + 8 * r) * S::kPieces * 16;
                        if constexpr (S::kWords == 4) {
                            const uint4 v = lds128(pw);
                            w[r][0] = v.x, w[r][1] = v.y, w[r][2] = v.z, w[r][3] = v.w;
                        } else if constexpr (S::kWords == 2) {
                            const uint2 v = lds64(pw);
                            w[r][0] = v.x, w[r][1] = v.y;
                        } else {
                            w[r][0] = lds32(pw);
                        }
                    }
                    const float s0 = half_of(sc[m][0], i), s1 = half_of(sc[m][1], i);
                    const float b0 = half_of(bi[m][0], i), b1 = half_of(bi[m][1], i);
#pragma unroll
                    for (int n = 0; n < kNT; ++n) {
                        float lo[4];
#pragma unroll
                        for (int p = 0; p < kParts; ++p) {
                            const uint4 v = x[n][p];
#pragma unroll
                            for (int h = 0; h < 2; ++h) {  // eight codes: one 4-bit word, two 8-bit ones
                                const int j = kBits == 4 ? 2 * h : 0;
                                const uint32_t w0 = w[0][kBits == 4 ? p : 2 * p + h], w1 = w[1][kBits == 4 ? p : 2 * p + h];
                                const uint32_t x0 = h ? v.z : v.x, x1 = h ? v.w : v.y;
                                const uint32_t f[4] = {codes2<kBits>(w0, j), codes2<kBits>(w1, j), codes2<kBits>(w0, j + 1),
                                                       codes2<kBits>(w1, j + 1)};
                                if (p == 0 && h == 0) mma16816_0(lo, f[0], f[1], f[2], f[3], x0, x1);
                                else mma16816(lo, f[0], f[1], f[2], f[3], x0, x1);
                            }
                        }
                        float(&o)[4] = y[m][n];
                        o[0] = fmaf(s0, lo[0] * xt[n].z, fmaf(b0, xt[n].x, o[0]));
                        o[1] = fmaf(s0, lo[1] * xt[n].w, fmaf(b0, xt[n].y, o[1]));
                        o[2] = fmaf(s1, lo[2] * xt[n].z, fmaf(b1, xt[n].x, o[2]));
                        o[3] = fmaf(s1, lo[3] * xt[n].w, fmaf(b1, xt[n].y, o[3]));
                    }
                }
            }
        }
        if (split == 1) {
#pragma unroll
            for (int m = 0; m < kMT; ++m)
#pragma unroll
                for (int n = 0; n < kNT; ++n)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int t = 8 * n + 2 * c + j % 2, o = tile * kRows + 16 * m + g + 8 * (j / 2);
                        if (t < nt && o < W.out) a.y[(int64_t)(t0 + t) * W.out + o] = f2bf16(y[m][n][j] * kBack);
                    }
            continue;
        }
        // the warps' parts, added in fixed order
        float* rb = red + buf * (kWarps * kRed);
#pragma unroll
        for (int m = 0; m < kMT; ++m)
#pragma unroll
            for (int n = 0; n < kNT; ++n)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    rb[warp * kRed + (8 * n + 2 * c + j % 2) * kRows + 16 * m + g + 8 * (j / 2)] = y[m][n][j];
        __syncthreads();
        for (int i = tid; i < across * nt * kRows; i += kThreads) {
            const int at = i / (nt * kRows), in = i % (nt * kRows);
            const int n = (tile - warp / split + at) * kRows + in % kRows;
            float v = 0.0f;
            for (int w = 0; w < split; ++w) v += rb[(at * split + w) * kRed + in];
            if (n < W.out) a.y[(int64_t)(t0 + in / kRows) * W.out + n] = f2bf16(v * kBack);
        }
    }
}

// Nibbles j and j + 4 of a word shifted by 4 j as the bf16 pair {128 + q_j, 128 + q_j+4}.
// (one three-input instruction: left to itself the compiler takes two)
__device__ __forceinline__ uint32_t nib2(uint32_t w) {
    uint32_t r;
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(w), "r"(0x000F000Fu), "r"(0x43004300u));
    return r;
}

// The matrix in bf16, one rounding per weight (the tensor core multiplies 16-bit operands, and the rows it meets are
// rounded to as many bits): eight codes, one 4-bit word or two 8-bit ones, to one 16-byte store, four of them a thread
// and step so that their loads are under way together.  Bound by the 2 bytes written per weight.
// Beside it, rows that TMA could not read (n values each, n no multiple of 8) are copied `pitch8` 16-byte pieces apart.
constexpr int kPieces = 4;
struct PadRows {
    const uint16_t* x;
    uint4* out;
    int64_t pieces;  // 0: none
    int n, pitch8;
};
template <int kBits>
__global__ void __launch_bounds__(256) dequant16_kernel(const moe_qtensor W, int64_t pieces, int shift, uint4* __restrict__ out,
                                                        const PadRows pad) {
    const int groups8 = W.group / 8;  // 1 << shift, or shift < 0
    grid_release();  // the product's blocks set themselves up meanwhile
    grid_wait();
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < pad.pieces; i += (int64_t)gridDim.x * 256) {
        const int64_t t = i / pad.pitch8;
        const int c = (int)(i - t * pad.pitch8) * 8;
        uint32_t v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = c + j < pad.n ? ld_after(pad.x + t * pad.n + c + j) : 0;
        pad.out[i] = make_uint4(v[0] | v[1] << 16, v[2] | v[3] << 16, v[4] | v[5] << 16, v[6] | v[7] << 16);
    }
    for (int64_t i0 = (int64_t)blockIdx.x * (256 * kPieces) + threadIdx.x; i0 < pieces;
         i0 += (int64_t)gridDim.x * (256 * kPieces)) {
        uint32_t w[kPieces][kBits / 4];
        uint16_t s[kPieces], b[kPieces];
#pragma unroll
        for (int j = 0; j < kPieces; ++j) {
            const int64_t i = i0 + j * 256;
            if (i >= pieces) break;
            if constexpr (kBits == 4) {
                w[j][0] = ld_after(W.packed + i);
            } else {
                const uint2 v = ld_after(reinterpret_cast<const uint2*>(W.packed) + i);
                w[j][0] = v.x, w[j][1] = v.y;
            }
            const int64_t g = shift >= 0 ? i >> shift : i / groups8;  // (a row is a whole number of groups)
            s[j] = ld_after(W.scales + g);
            b[j] = ld_after(W.biases + g);
        }
#pragma unroll
        for (int j = 0; j < kPieces; ++j) {
            const int64_t i = i0 + j * 256;
            if (i >= pieces) break;
            const __nv_bfloat162 s2 = __bfloat162bfloat162(__ushort_as_bfloat16(s[j]));
            const __nv_bfloat162 b2 = __bfloat162bfloat162(__ushort_as_bfloat16(b[j]));
            const __nv_bfloat162 k128 = __float2bfloat162_rn(128.0f);
            auto nib = [&](uint32_t v) {  // the low nibbles of bytes 0 and 2 (exact)
                const uint32_t r = nib2(v);
                return __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&r), k128);
            };
            auto affine = [&](__nv_bfloat162 q) {
                const __nv_bfloat162 d = __hfma2(q, s2, b2);
                return *reinterpret_cast<const uint32_t*>(&d);
            };
            uint32_t o[4];
            if constexpr (kBits == 4) {  // pairs (0, 4) (1, 5) (2, 6) (3, 7)
                uint32_t d[4];
#pragma unroll
                for (int h = 0; h < 4; ++h) d[h] = affine(nib(w[j][0] >> (4 * h)));
                o[0] = __byte_perm(d[0], d[1], 0x5410), o[1] = __byte_perm(d[2], d[3], 0x5410);
                o[2] = __byte_perm(d[0], d[1], 0x7632), o[3] = __byte_perm(d[2], d[3], 0x7632);
            } else {                     // a word: (0, 2) (1, 3); bf16 holds every whole number up to 256
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint32_t x = w[j][h];
                    const __nv_bfloat162 k16 = __float2bfloat162_rn(16.0f);
                    const uint32_t d0 = affine(__hfma2(nib(x >> 4), k16, nib(x)));
                    const uint32_t d1 = affine(__hfma2(nib(x >> 12), k16, nib(x >> 8)));
                    o[2 * h] = __byte_perm(d0, d1, 0x5410), o[2 * h + 1] = __byte_perm(d0, d1, 0x7632);
                }
            }
            out[i] = make_uint4(o[0], o[1], o[2], o[3]);
        }
    }
}

// The parts of split sums, added in order and rounded once.
__global__ void __launch_bounds__(256) add_parts_kernel(const float* __restrict__ parts, int splits, int64_t n,
                                                        uint16_t* __restrict__ y) {
    grid_wait();
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
        float v = 0.0f;
#pragma unroll 8
        for (int s = 0; s < splits; ++s) v += ld_after(parts + s * n + i);
        y[i] = f2bf16(v);
    }
}

template <int kBits, int kUnit>
size_t codes_smem(const moe_qtensor& W, int tb, int mt) {
    const size_t ring = mt == 2 ? Slot<kBits, kUnit, 2>::kDepth * Slot<kBits, kUnit, 2>::kBytes
                                : Slot<kBits, kUnit, 1>::kDepth * Slot<kBits, kUnit, 1>::kBytes;
    return kWarps * ring + (size_t)tb * W.in * 2 + kUnit * 2 + (size_t)(W.in / kUnit) * ((tb + 1) & ~1) * 8 + 16 +
           2u * kWarps * (tb > 8 ? 16 : 8) * 16 * mt * sizeof(float);
}

template <int kBits, int kUnit, int kNT, int kMT, int kVec>
cudaError_t launch_vec(LinArgs a, cudaStream_t s) {
    const size_t smem = codes_smem<kBits, kUnit>(a.W, a.block, kMT);
    static SmemLimit limit;
    constexpr auto kernel = linear_codes_kernel<kBits, kUnit, kNT, kMT, kVec>;
    const cudaError_t e = limit.raise((const void*)kernel, kMaxSmem);
    if (e != cudaSuccess) return e;
    constexpr int kRows = 16 * kMT;
    const int tiles = (a.W.out + kRows - 1) / kRows, across = (a.T + a.block - 1) / a.block;
    const int room = std::max(1, (smem > 112 * 1024 ? 1 : 2) * device_sms() / across);
    // The warps that share a tile (1, 2, 4 or 8): the fewest rounds' worth of quads a warp walks, a round of shared
    // tiles costing about a quarter of a quad more for adding the parts up.  (2048 inputs, one token: 131072 outputs
    // take 36.6 us with four warps, 39.6 with one, whose second round is three quarters empty; 512 outputs need all
    // eight.)
    const int quads = (a.units + kQuad - 1) / kQuad;
    int64_t best = INT64_MAX;
    for (int s = 1; s <= kWarps && s <= std::max(quads, 1); s *= 2) {
        const int64_t at_once = (int64_t)room * (kWarps / s);
        const int64_t cost = (tiles + at_once - 1) / at_once * (4 * ((quads + s - 1) / s) + (s > 1));
        if (cost < best) best = cost, a.split = s;
    }
    const int per = kWarps / a.split, want = (tiles + per - 1) / per;
    return launch_dependent(kernel, dim3(std::min(want, room), across), kThreads, smem, 1, s, a);
}

template <int kBits, int kUnit, int kNT, int kMT>
cudaError_t launch_codes(const LinArgs& a, cudaStream_t s) {
    const bool vec = a.W.group == kUnit && a.units % kQuad == 0 && (((uintptr_t)a.W.scales | (uintptr_t)a.W.biases) & 7) == 0;
    return vec ? launch_vec<kBits, kUnit, kNT, kMT, 1>(a, s) : launch_vec<kBits, kUnit, kNT, kMT, 0>(a, s);
}

template <int kBits, int kUnit>
cudaError_t launch_unit(LinArgs a, cudaStream_t s) {
    a.units = a.W.in / kUnit;
    const uint32_t span = a.W.group / kUnit;
    a.inv_span = span > 1 ? (uint32_t)(((1ull << 32) + span - 1) / span) : 0;
    const int chunks = a.W.in / 8;
    a.inv_chunks = (uint32_t)(((1ull << 32) + chunks - 1) / chunks);
    a.step_t = kThreads / chunks;
    a.step_c = kThreads % chunks;
    // as many tokens a block as one or two token tiles hold and shared memory takes
    int tb = std::min(a.T, 16);
    while (tb > 1 && codes_smem<kBits, kUnit>(a.W, tb, 1) > kMaxSmem) --tb;
    const int blocks = (a.T + tb - 1) / tb;
    a.block = (a.T + blocks - 1) / blocks;
    if (a.block > 8) return launch_codes<kBits, kUnit, 2, 1>(a, s);
    // tall matrices: two row tiles a warp share the loads of x (and two blocks still fit an SM)
    if (a.W.out >= 32 * 2 * kWarps * device_sms() && codes_smem<kBits, kUnit>(a.W, a.block, 2) <= 112 * 1024)
        return launch_codes<kBits, kUnit, 1, 2>(a, s);
    return launch_codes<kBits, kUnit, 1, 1>(a, s);
}

}  // namespace

// Whether a row of x, and the ring beside it, fit in shared memory (from about 54,000 8-bit inputs on they do not).
bool affine_codes_supported(const moe_qtensor& W) {
    const size_t smem = W.group % 64 == 0 ? (W.bits == 4 ? codes_smem<4, 64>(W, 1, 1) : codes_smem<8, 64>(W, 1, 1))
                                          : (W.bits == 4 ? codes_smem<4, 32>(W, 1, 1) : codes_smem<8, 32>(W, 1, 1));
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

namespace {
unsigned blocks_for(int64_t n) { return (unsigned)std::min<int64_t>((n + 255) / 256, (int64_t)device_sms() * 8); }
}  // namespace

cudaError_t launch_affine_dequant16(const moe_qtensor& W, uint16_t* out, const uint16_t* rows, int T, int n,
                                    uint16_t* padded, cudaStream_t s) {
    const int64_t pieces = (int64_t)W.out * W.in / 8;
    int shift = 0;
    while (8 << shift < W.group) ++shift;
    if (8 << shift != W.group) shift = -1;
    PadRows pad = {};
    if (padded) pad = {rows, reinterpret_cast<uint4*>(padded), (int64_t)T * ((n + 7) / 8), n, (n + 7) / 8};
    const unsigned blocks = std::max(blocks_for((pieces + kPieces - 1) / kPieces), blocks_for(pad.pieces));
    return launch_dependent(W.bits == 4 ? dequant16_kernel<4> : dequant16_kernel<8>, dim3(blocks), 256, 0, 1, s, W, pieces,
                            shift, reinterpret_cast<uint4*>(out), pad);
}

cudaError_t launch_add_parts(const float* parts, int splits, int64_t n, uint16_t* y, cudaStream_t s) {
    return launch_dependent(add_parts_kernel, dim3(blocks_for(n)), 256, 0, 1, s, parts, splits, n, y);
}

}  // namespace moeq
