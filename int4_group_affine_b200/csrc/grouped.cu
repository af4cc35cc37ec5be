// grouped.cu - products grouped by expert with ragged sizes, and their gradients, on warp-level
// tensor-core tiles: the kernel that takes every size and alignment.  Operands whose rows are whole
// 16-byte pieces go to the tcgen05 kernel (grouped_tc.cu) instead; TMA cannot read others.
//
// A block owns a 128 x 128 tile of the output and steps through the sum 32 terms at a time.  Rows may
// start at any element, so the aligned 16-byte pieces that they lie in are copied as they are
// (cp.async, four steps ahead: the copies' latency is what a block with few tiles beside it waits
// for), and on their way from there to the tile the elements are shifted into place (a row's shift
// is the same in every step, which advances by 64 bytes or by 32 whole rows) and whatever lies outside
// the matrix or, for the weight gradient, outside the group's rows becomes zero, so a NaN in another
// group's row never meets a sum.  No byte outside the tensors is read.  Eight warps of 64 x 32 run
// mma.sync m16n8k16 (fp32 accumulators) on the tile.  An operand whose terms are contiguous in memory
// is kept [row][term], one whose rows are, [term][row], which ldmatrix transposes; pitches of 80 and
// 272 bytes put the eight rows of an ldmatrix in different banks.
//
// Bound by the instructions that fetch, shift and place the operands (a step of a lone block takes 2500
// cycles: copies 500 to 800, shifting 1000 to 1400, products 800) and by the warp-level tensor path
// (about a quarter of tcgen05's rate): 7500 rows on 16 experts of 1003 to 1001, forward 145 us (104 TFLOP/s;
// with 2-byte loads into 64 x 64 tiles 369), row gradient 135, weight gradient 129, to fp32 157.
#include <cuda_fp16.h>

#include "grouped.cuh"

namespace moeq {
namespace {

constexpr int kT = 128, kKT = 32, kThreads = 256, kAhead = 4;
constexpr int kPitchT = kKT + 8;  // [row][term]
constexpr int kPitchR = kT + 8;   // [term][row]
// The tensor core's fp32 accumulation rounds toward zero, an error that grows with the length of the
// sum (measured 4.7e-7 of the result at 512 terms, 9.1e-6 at 8192); longer sums for fp32 results, and those that may be
// longer than kLong16 terms for 16-bit ones, are added up in parts of this length with rounded fp32 additions.
constexpr int kPart = 512, kLong16 = 8192;

template <int kF16>
__device__ __forceinline__ void mma16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if (kF16)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, "
            "%2, %3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, "
            "%1, %2, %3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <int kTrans>
__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], const uint16_t* p) {
    const uint32_t a = (uint32_t)__cvta_generic_to_shared(p);
    if (kTrans)
        asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                     : "r"(a)
                     : "memory");
    else
        asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                     : "r"(a)
                     : "memory");
}

template <int kF16>
__device__ __forceinline__ uint16_t to16(float v) {
    return kF16 ? __half_as_ushort(__float2half_rn(v)) : f2bf16(v);
}
template <int kF16>
__device__ __forceinline__ float from16(uint16_t v) {
    return kF16 ? __half2float(__ushort_as_half(v)) : bf16f(v);
}

__device__ __forceinline__ void cp16(uint32_t dst, const void* src, int bytes) {  // (the rest of the 16: zeros)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}

// 16 whole bytes where `on`, without a branch.
__device__ __forceinline__ void cp16_if(uint32_t dst, const void* src, uint32_t on) {
    asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %2, 0;\n\t@q cp.async.cg.shared.global [%0], [%1], 16;\n\t}" ::"r"(dst),
                 "l"(src), "r"(on)
                 : "memory");
}

// Eight 16-bit elements out of the two aligned pieces they lie in, from byte `off` on; the first n count.
__device__ __forceinline__ uint4 shifted(const uint4& lo, const uint4& hi, int off, int n) {
    uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
    if (off & 8) {
#pragma unroll
        for (int i = 0; i < 6; ++i) w[i] = w[i + 2];
    }
    if (off & 4) {
#pragma unroll
        for (int i = 0; i < 5; ++i) w[i] = w[i + 1];
    }
    if (off & 2) {
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = __funnelshift_r(w[i], w[i + 1], 16);
    }
    if (n < 8) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (2 * i + 1 >= n) w[i] &= 0xFFFFu;
            if (2 * i >= n) w[i] = 0;
        }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// A piece that may reach outside the tensor [first, last).
__device__ __noinline__ void copy_edge(unsigned char* dst, const char* src, const uint16_t* first, const uint16_t* last) {
    const char *begin = reinterpret_cast<const char*>(first), *end = reinterpret_cast<const char*>(last);
    if (src >= begin) {
        const int bytes = (int)min((int64_t)16, max((int64_t)0, (int64_t)(end - src)));
        const uintptr_t from = reinterpret_cast<uintptr_t>(bytes ? src : begin) & ~(uintptr_t)15;  // (an aligned one even for none)
        cp16((uint32_t)__cvta_generic_to_shared(dst), reinterpret_cast<const void*>(from), bytes);
    } else {  // the tensor begins inside the piece
        for (int b = (int)(begin - src); b < 16 && src + b < end; b += 2)
            *reinterpret_cast<uint16_t*>(dst + b) = ld_after(reinterpret_cast<const uint16_t*>(src + b));
    }
}

// One operand of the tile: 128 rows x 32 terms a step.  kRows: the rows are contiguous in memory (else the terms).  A
// line is what is contiguous of a step: a row's 32 terms, or a term's 128 rows.
template <int kRows>
struct Operand {
    static constexpr int kElems = kRows ? kKT * kPitchR : kT * kPitchT;
    static constexpr int kLines = kRows ? kKT : kT, kEights = kRows ? kT / 8 : kKT / 8;
    static constexpr int kPieces = kEights + 1;              // aligned pieces a line lies in
    static constexpr int kRaw = kLines * kPieces * 16;       // bytes of a step
    const uint16_t *p, *first, *last;  // the group's first element; the tensor
    int64_t ld;
    int row0, rows, terms;

    __device__ __forceinline__ const uint16_t* line(int t0, int i) const {
        return kRows ? p + (int64_t)(t0 + i) * ld + row0 : p + (int64_t)(row0 + i) * ld + t0;
    }
    __device__ __forceinline__ bool live(int t0, int i) const { return kRows ? t0 + i < terms : row0 + i < rows; }

    // What stays the same from step to step, for this thread's pieces and eights: where they are, and whether a whole
    // step's are all inside the tensor.
    static constexpr int kCopies = (kLines * kPieces + kThreads - 1) / kThreads, kPlaces = kLines * kEights / kThreads;
    const char* src[kCopies];
    uint32_t safe;  // bit h: piece h of every whole step is inside the tensor
    bool easy;      // every piece of the warp is that, or of a dead line
    int off[kPlaces], count[kPlaces];

    __device__ __forceinline__ void start(int tid) {
        const int64_t steps = terms / kKT;  // whole ones
        bool edge = false;
        safe = 0;
#pragma unroll
        for (int h = 0; h < kCopies; ++h) {
            const int i = tid + h * kThreads, l = min(i / kPieces, kLines - 1);
            src[h] = reinterpret_cast<const char*>(reinterpret_cast<uintptr_t>(line(0, l)) & ~(uintptr_t)15) + i % kPieces * 16;
            if (i >= kLines * kPieces || steps == 0 || !(kRows || live(0, l))) continue;
            if (src[h] >= reinterpret_cast<const char*>(first) &&
                src[h] + (steps - 1) * (kRows ? ld * (2 * kKT) : 2 * kKT) + 16 <= reinterpret_cast<const char*>(last))
                safe |= 1u << h;
            else
                edge = true;
        }
        easy = !__any_sync(0xffffffffu, edge);
#pragma unroll
        for (int h = 0; h < kPlaces; ++h) {
            const int i = tid + h * kThreads, l = i / kEights;
            off[h] = (int)(reinterpret_cast<uintptr_t>(line(0, l)) & 15);
            count[h] = kRows ? min(max(rows - (row0 + i % kEights * 8), 0), 8) : live(0, l) ? 8 : 0;
        }
    }
    __device__ __forceinline__ void copy(unsigned char* raw, int t0, int tid) {
        const bool whole = t0 + kKT <= terms;
        const uint32_t dst0 = (uint32_t)__cvta_generic_to_shared(raw) + tid * 16;
        if (whole && easy) {
#pragma unroll
            for (int h = 0; h < kCopies; ++h) {
                cp16_if(dst0 + h * kThreads * 16, src[h], safe >> h & 1);
                src[h] += kRows ? ld * (2 * kKT) : 2 * kKT;
            }
            return;
        }
#pragma unroll
        for (int h = 0; h < kCopies; ++h) {
            if (whole && (safe >> h & 1)) cp16(dst0 + h * kThreads * 16, src[h], 16);
            else if (tid + h * kThreads < kLines * kPieces && live(t0, (tid + h * kThreads) / kPieces))
                copy_edge(raw + (tid + h * kThreads) * 16, src[h], first, last);
            src[h] += kRows ? ld * (2 * kKT) : 2 * kKT;  // (32 rows are whole pieces whatever their length)
        }
    }
    __device__ __forceinline__ void place(uint16_t* s, const unsigned char* raw, int t0, int tid) const {
        const bool whole = t0 + kKT <= terms;
#pragma unroll
        for (int h = 0; h < kPlaces; ++h) {
            const int i = tid + h * kThreads, l = i / kEights, c = i % kEights;
            int n = count[h];
            if (!whole) n = kRows ? (live(t0, l) ? n : 0) : min(n, max(terms - (t0 + c * 8), 0));
            const uint4* at = reinterpret_cast<const uint4*>(raw) + l * kPieces + c;
            uint4 v = make_uint4(0, 0, 0, 0);
            if (n > 0) v = shifted(at[0], at[1], off[h], n);
            *reinterpret_cast<uint4*>(s + l * (kRows ? kPitchR : kPitchT) + c * 8) = v;
        }
    }
    // mma.sync's A fragment of rows [r, r + 16), terms [k, k + 16)
    __device__ __forceinline__ static void frag_a(uint32_t (&f)[4], const uint16_t* s, int r, int k, int lane) {
        const int q = lane / 8, l = lane % 8;
        if (kRows) ldmatrix4<1>(f, s + (k + q / 2 * 8 + l) * kPitchR + r + q % 2 * 8);
        else ldmatrix4<0>(f, s + (r + q % 2 * 8 + l) * kPitchT + k + q / 2 * 8);
    }
    // and two B fragments (b0, b1 of rows [r, r + 8), then of [r + 8, r + 16))
    __device__ __forceinline__ static void frag_b(uint32_t (&f)[4], const uint16_t* s, int r, int k, int lane) {
        const int q = lane / 8, l = lane % 8;
        if (kRows) ldmatrix4<1>(f, s + (k + q % 2 * 8 + l) * kPitchR + r + q / 2 * 8);
        else ldmatrix4<0>(f, s + (r + q / 2 * 8 + l) * kPitchT + k + q % 2 * 8);
    }
};

__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// A float of the cluster's block `rank`, at this block's shared memory address `addr`.
__device__ __forceinline__ float ld_of(uint32_t addr, int rank) {
    float v;
    asm volatile("{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %1, %2;\n\tld.shared::cluster.f32 %0, [a];\n\t}"
                 : "=f"(v)
                 : "r"(addr), "r"(rank)
                 : "memory");
    return v;
}

// kParts: sums in parts.  kSplit: a cluster's a.splits blocks share a tile's sum (weight gradients).
template <int kDir, int kF16, int kParts, int kSplit>
__global__ void __launch_bounds__(kThreads, kParts ? 1 : 2) gmm_any_kernel(const GmmArgs a) {
    using A = Operand<kDir == kGmmDw>;
    using B = Operand<kDir != kGmmFwd>;
    extern __shared__ __align__(16) unsigned char sm[];  // [steps ahead][A, B], then the tile
    constexpr int kRaw = A::kRaw + B::kRaw;
    uint16_t *sA = reinterpret_cast<uint16_t*>(sm + kAhead * kRaw), *sB = sA + A::kElems;
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32, g8 = lane / 4, c4 = lane % 4;
    grid_wait();
    if (blockIdx.x == 0) (void)gmm_check_offsets(a, tid, kThreads);

    // the tile: group, output rows [i0, I) and columns [j0, J), terms [0, S)
    const int J = kDir == kGmmFwd ? a.N : a.K;
    const int jt = (J + kT - 1) / kT;
    int g, i0, j0, I, S;
    GmmRows rows;
    const int rank = kSplit ? blockIdx.x % a.splits : 0;
    if (kDir == kGmmDw) {
        const int it = (a.N + kT - 1) / kT, tile = kSplit ? blockIdx.x / a.splits : blockIdx.x;
        g = (int)(tile / ((int64_t)it * jt));
        const int rem = (int)(tile % ((int64_t)it * jt));
        rows = gmm_rows_of(a, g, lane);
        if (kSplit) {  // this block's rows, whole steps
            const int steps = (rows.end - rows.begin + kKT - 1) / kKT, per = (steps + a.splits - 1) / a.splits * kKT;
            rows.begin = min(rows.begin + rank * per, rows.end);
            rows.end = min(rows.begin + per, rows.end);
        }
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
    const int la = kDir == kGmmFwd ? a.K : a.N;  // a row of the first operand
    A oa;
    oa.first = a.a;
    oa.last = a.a + (int64_t)a.M * la;
    oa.p = a.a + (int64_t)rows.begin * la;
    oa.ld = la;
    oa.row0 = i0;
    oa.rows = I;
    oa.terms = S;
    B ob;
    ob.first = a.b;
    ob.last = a.b + (kDir == kGmmDw ? (int64_t)a.M * a.K : a.G * nk);
    ob.p = kDir == kGmmDw ? a.b + (int64_t)rows.begin * a.K : a.b + g * nk;
    ob.ld = a.K;
    ob.row0 = j0;
    ob.rows = J;
    ob.terms = S;

    float acc[4][4][4], sum[kParts ? 4 : 1][4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                acc[i][j][q] = 0.0f;
                if (kParts) sum[kParts ? i : 0][j][q] = 0.0f;
            }

    const int wi = warp / 4 * 64, wj = warp % 4 * 32;
    oa.start(tid);
    ob.start(tid);
    auto copy = [&](int t0) {
        if (t0 < S) {
            unsigned char* raw = sm + t0 / kKT % kAhead * kRaw;
            oa.copy(raw, t0, tid);
            ob.copy(raw + A::kRaw, t0, tid);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
#pragma unroll
    for (int h = 0; h < kAhead - 1; ++h) copy(h * kKT);
    for (int t0 = 0; t0 < S; t0 += kKT) {
        asm volatile("cp.async.wait_group %0;" ::"n"(kAhead - 2) : "memory");
        __syncthreads();  // the step's pieces are there, and the tile and the step before's pieces are read
        copy(t0 + (kAhead - 1) * kKT);
        const unsigned char* raw = sm + t0 / kKT % kAhead * kRaw;
        oa.place(sA, raw, t0, tid);
        ob.place(sB, raw + A::kRaw, t0, tid);
        __syncthreads();
#pragma unroll
        for (int ks = 0; ks < kKT; ks += 16) {
            uint32_t fb[2][4];
#pragma unroll
            for (int j = 0; j < 2; ++j) B::frag_b(fb[j], sB, wj + 16 * j, ks, lane);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                uint32_t fa[4];
                A::frag_a(fa, sA, wi + 16 * i, ks, lane);
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    mma16<kF16>(acc[i][j], fa, fb[j / 2][j % 2 * 2], fb[j / 2][j % 2 * 2 + 1]);
            }
        }
        if (kParts && ((t0 + kKT) % kPart == 0 || t0 + kKT >= S)) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j)
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        sum[kParts ? i : 0][j][q] += acc[i][j][q];
                        acc[i][j][q] = 0.0f;
                    }
        }
    }

    const int64_t out0 = kDir == kGmmDw ? g * nk : (int64_t)rows.begin * J;
    auto store = [&](int i, int j, int q, float v) {
        const int r = i0 + wi + 16 * i + g8 + 8 * (q / 2), c = j0 + wj + 8 * j + 2 * c4 + q % 2;
        if (r >= I || c >= J) return;
        const int64_t at = out0 + (int64_t)r * J + c;
        if (kParts && a.out_f32) {
            float* o = reinterpret_cast<float*>(a.out) + at;
            *o = a.accumulate ? *o + v : v;
        } else {
            uint16_t* o = reinterpret_cast<uint16_t*>(a.out) + at;
            if (kDir == kGmmDw && a.accumulate) v += from16<kF16>(*o);
            *o = to16<kF16>(v);
        }
    };
    float* sv = reinterpret_cast<float*>(sm);  // kSplit: [value of a thread][thread], over the copies
    if (kSplit) {
        asm volatile("cp.async.wait_all;" ::: "memory");
        __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const float v = kParts ? sum[kParts ? i : 0][j][q] : acc[i][j][q];
                if (kSplit) sv[((i * 4 + j) * 4 + q) * kThreads + tid] = v;
                else store(i, j, q, v);
            }
    if (kSplit) {  // every block adds up its share of the values, in the blocks' order
        static_assert(64 * kThreads * 4 <= kAhead * kRaw, "the values take the copies' place");
        cluster_sync();
        const uint32_t base = (uint32_t)__cvta_generic_to_shared(sv + tid);
        const int share = 64 / a.splits;
        for (int e = rank * share; e < (rank + 1) * share; ++e) {
            float part[8], v = 0.0f;
#pragma unroll
            for (int b = 0; b < 8; ++b) part[b] = b < a.splits ? ld_of(base + e * (kThreads * 4), b) : 0.0f;
#pragma unroll
            for (int b = 0; b < 8; ++b) v += part[b];
            store(e / 16, e / 4 % 4, e % 4, v);
        }
        cluster_sync();  // (no block ends while another reads it)
    }
}

template <int kDir, int kF16, int kParts, int kSplit>
cudaError_t launch_parts(const GmmArgs& a, unsigned tiles, cudaStream_t s) {
    using A = Operand<kDir == kGmmDw>;
    using B = Operand<kDir != kGmmFwd>;
    constexpr size_t smem = kAhead * (A::kRaw + B::kRaw) + (A::kElems + B::kElems) * 2;
    static_assert(2 * smem <= 227 * 1024 - 2048, "two blocks a multiprocessor");
    static SmemLimit limit;
    constexpr auto kernel = gmm_any_kernel<kDir, kF16, kParts, kSplit>;
    const cudaError_t e = limit.raise((const void*)kernel, smem);
    if (e != cudaSuccess) return e;
    const int cluster = kSplit ? a.splits : 1;
    return launch_dependent(kernel, dim3(tiles * cluster), kThreads, smem, cluster, s, a);
}

template <int kDir, int kF16>
cudaError_t launch_any(const GmmArgs& a, cudaStream_t s) {
    const int64_t jt = ((kDir == kGmmFwd ? a.N : a.K) + kT - 1) / kT;
    // forward and dx: a group's last tile may be partly filled, so at most one more per group
    const int64_t tiles = kDir == kGmmDw ? (int64_t)a.G * ((a.N + kT - 1) / kT) * jt
                                         : ((int64_t)a.M / kT + (a.off ? a.G : 1)) * jt;
    if (tiles > INT32_MAX) return cudaErrorInvalidConfiguration;
    if constexpr (kDir == kGmmDw)
        if (a.splits > 1) return launch_parts<kDir, kF16, 1, 1>(a, (unsigned)tiles, s);
    if ((kDir == kGmmDw && a.out_f32) || (kDir == kGmmFwd ? a.K : kDir == kGmmDx ? a.N : a.M) > kLong16)
        return launch_parts<kDir, kF16, 1, 0>(a, (unsigned)tiles, s);
    return launch_parts<kDir, kF16, 0, 0>(a, (unsigned)tiles, s);
}

// Weight gradients of few tiles and many rows (adapter factors): as many blocks as would be idle, up to eight, share a
// tile's rows, at least 128 rows of the average group each (4000 rows, 3 experts of 51 x 75: 15.7 us, one block a tile 75;
// 1200 rows of 500 x 333: 13.6 and 54).
int dw_splits(const GmmArgs& a) {
    const int64_t tiles = (int64_t)a.G * ((a.N + kT - 1) / kT) * ((a.K + kT - 1) / kT);
    int splits = 8;
    while (splits > 1 && (tiles * splits > device_sms() || a.M / a.G < 128 * splits)) splits /= 2;
    return splits;
}

}  // namespace

cudaError_t launch_grouped(int dir, int f16, const GmmArgs& a, cudaStream_t s) {
    if (grouped_tc_supported(dir, a)) return launch_grouped_tc(dir, f16, a, 0, s);
    if (dir == kGmmDw) {
        GmmArgs b = a;
        b.splits = dw_splits(a);
        return f16 ? launch_any<kGmmDw, 1>(b, s) : launch_any<kGmmDw, 0>(b, s);
    }
    if (dir == kGmmFwd) return f16 ? launch_any<kGmmFwd, 1>(a, s) : launch_any<kGmmFwd, 0>(a, s);
    return f16 ? launch_any<kGmmDx, 1>(a, s) : launch_any<kGmmDx, 0>(a, s);
}

}  // namespace moeq
