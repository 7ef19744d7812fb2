// grouped_stream.hpp -- expert products with few rows an expert: C[r] = A[r] .
// B[g], bound by the bytes of the experts' weights.
//
// The weights go from HBM straight to registers, every byte once per 16 rows, and
// no LDS lies between: at a few rows a weight is used by a single matrix
// instruction.  A workgroup takes a strip of columns of one expert, its waves
// split K stage by stage, and their sums are added in LDS in wave order.
// The weights are the matrix instruction's first operand and the tokens its
// second, so that a lane holds neighbouring columns of one row of C.
//
// A stage is eight 16-byte loads a lane (8 KiB a wave), twice in flight:
//  * B as stored (n contiguous): lane l = 16 g + c loads, of 16-bit types, the
//    rows k = 8 g .. 8 g + 7 at the columns 8 c .. 8 c + 7, an 8 x 8 square that
//    it transposes in registers: fragment j is column 8 c + j.  128 columns by 32
//    k.  fp32 needs no transpose: of 16 k, rows 4 g .. 4 g + 3 at columns 4 c ..
//    4 c + 3; element j of row e feeds instruction e of fragment j.  64 by 32.
//  * B transposed (k contiguous): a load is a fragment, row n = 16 j + c, a
//    16-byte chunk of k at lane group g.  32 columns by 128 k (fp32: 64 k).
// Measured: 32 rows over 7 of 8 experts of 1024 x 4096 bf16 12.4 us (4.7 TB/s of weights).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "expert_rows.hpp"

namespace tg {

struct GroupedParams {
    const char *A, *B;
    char *C;
    const int32_t *offsets;
    int64_t lda, ldb, ldc, sB, sC;      // sC: wgrad only
    int experts, rows;
    int M, N, K;                         // wgrad: C[g] is M x N (K unused); grouped: rows x N over K
    int c_f32;
    // C stored past the caches: set where operands and result together exceed the
    // 256 MiB last-level cache, in which a result would then drive out operands that
    // other workgroups still read (16384 x 4096 x 2048 bf16 over 8 experts: forward 245 ->
    // 229 us, the gradients 245 -> 234 and 249 -> 222; where all of it fits, the hint costs:
    // 8192 x 8192 x 2048 for one expert 211 -> 213 us).
    int past;
};

template <int DT, bool TRANS>
struct StreamShape {
    static constexpr int E = DT == DT_F32 ? 4 : 2, PER = 16 / E;
    static constexpr int FRAGS = TRANS ? 2 : PER;                    // column fragments of 16
    static constexpr int COLS = 16 * FRAGS;
    static constexpr int K = TRANS ? 16 * E == 64 ? 64 : 128 : 32;   // k of a stage
    static constexpr int A_LOADS = K / (4 * PER);                    // 16-byte loads of a row of A
};

template <int DT, bool TRANS>
struct StreamB {
    using S = StreamShape<DT, TRANS>;
    u32x4 q[8];
    // How much of a stage exists: all of it, whole 16-byte chunks, or any elements.
    enum Part { ALL = 0, CHUNKS = 1, ELEMENTS = 2 };
    template <int PART>
    __device__ __forceinline__ void load(const char *B, int64_t ldb, int n_left, int k_left, int lane) {
        const rsrc_t r = make_rsrc(B);
        const int g = lane / 16, c = lane % 16, ld = (int)ldb;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            int k, n, left;      // first element, elements there along the contiguous axis
            if constexpr (TRANS) {
                n = 16 * (i / 4) + c;
                k = 4 * S::PER * (i % 4) + S::PER * g;
                left = n < n_left ? k_left - k : 0;
            } else {
                n = S::PER * c;
                k = DT == DT_F32 ? 16 * (i / 4) + 4 * g + i % 4 : 8 * g + i;
                left = k < k_left ? n_left - n : 0;
            }
            const int at = (TRANS ? n * ld + k : k * ld + n) * S::E;
            if constexpr (PART == ALL) {
                // one lane offset for every load, the rest scalar
                const int i0 = (TRANS ? c * ld + S::PER * g : (DT == DT_F32 ? 4 : 8) * g * ld + S::PER * c) * S::E;
                const int step = TRANS ? 16 * (i / 4) * ld + 4 * S::PER * (i % 4)
                                       : (DT == DT_F32 ? 16 * (i / 4) + i % 4 : i) * ld;
                q[i] = bload16(r, i0, step * S::E);
            }
            else if constexpr (PART == CHUNKS) {
                q[i] = bload16(r, left > 0 ? at : kOutOfRange, 0);
            } else {
                // its address made here: the addresses of every chunk's elements, which the
                // stage does not change, would otherwise be held through the loop
                int here = left > 0 ? at : kOutOfRange;
                asm volatile("" : "+v"(here));
                q[i] = bload16_n<S::E>(r, here, 0, left < 0 ? 0 : left);
            }
        }
    }
};

// rows of A: A_LOADS chunks of this lane's row of 16
template <int DT, bool TRANS>
struct StreamA {
    using S = StreamShape<DT, TRANS>;
    u32x4 a[S::A_LOADS];
    template <int PART>
    __device__ __forceinline__ void load(const char *A, int64_t lda, int rows, int k_left, int lane) {
        const rsrc_t r = make_rsrc(A);
        const int g = lane / 16;
        const int row = lane % 16;
#pragma unroll
        for (int s = 0; s < S::A_LOADS; ++s) {
            const int k = 4 * S::PER * s + S::PER * g;
            const int at = row < rows ? (row * (int)lda + k) * S::E : kOutOfRange;
            const int left = row < rows ? k_left - k : 0;
            if constexpr (PART == StreamB<DT, TRANS>::ALL) {
                a[s] = bload16(r, at, 0);
            } else if constexpr (PART == StreamB<DT, TRANS>::CHUNKS) {
                a[s] = bload16(r, left > 0 ? at : kOutOfRange, 0);
            } else {
                int here = at;
                asm volatile("" : "+v"(here));
                a[s] = bload16_n<S::E>(r, here, 0, left < 0 ? 0 : left);
            }
        }
    }
};

template <int DT, bool TRANS>
__device__ __forceinline__ void stream_mma(const StreamB<DT, TRANS> &b, const StreamA<DT, TRANS> &a,
                                           f32x4 (&acc)[StreamShape<DT, TRANS>::FRAGS]) {
    using S = StreamShape<DT, TRANS>;
    if constexpr (DT == DT_F32) {
#pragma unroll
        for (int s = 0; s < S::A_LOADS; ++s)
#pragma unroll
            for (int e = 0; e < 4; ++e)
#pragma unroll
                for (int j = 0; j < S::FRAGS; ++j) {
                    const uint32_t w = TRANS ? b.q[4 * j + s][e] : b.q[4 * s + e][j], x = a.a[s][e];
                    acc[j] = __builtin_amdgcn_mfma_f32_16x16x4f32(__builtin_bit_cast(float, w),
                                                                 __builtin_bit_cast(float, x), acc[j], 0, 0, 0);
                }
    } else if constexpr (TRANS) {
#pragma unroll
        for (int s = 0; s < 4; ++s)
#pragma unroll
            for (int j = 0; j < 2; ++j) mfma_chunk<DT>(b.q[4 * j + s], a.a[s], acc[j]);
    } else {
        u32x4 f[8];
        transpose_square<2>(b.q, f);
#pragma unroll
        for (int j = 0; j < 8; ++j) mfma_chunk<DT>(f[j], a.a[0], acc[j]);
    }
}

// grid: column strips x row tiles (row_slot), at the same time; an expert's further row
// tiles read its weights again, from cache.
template <int DT, bool TRANS>
__global__ __launch_bounds__(512) void grouped_stream_kernel(GroupedParams p) {
    using S = StreamShape<DT, TRANS>;
    extern __shared__ f32x4 stream_lds[];           // [waves][FRAGS][64]
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int lane = threadIdx.x & 63, waves = blockDim.x >> 6;
    const int n0 = blockIdx.x * S::COLS;
    const int n_left = p.N - n0;
    const bool wide = p.ldc % 4 == 0 && reinterpret_cast<uintptr_t>(p.C) % 16 == 0;
    const int64_t b_step = (TRANS ? (int64_t)S::K : S::K * p.ldb) * S::E;
    int e;
    RowSpan span;
    if (!row_slot<16>(p.offsets, p.experts, p.rows, slot_of(p.experts), e, span)) return;
    const int r0 = span.lo, rows = span.hi - r0;
    const int stages = e == p.experts ? 0 : (p.K + S::K - 1) / S::K;
    const char *B = p.B + (e == p.experts ? 0 : (int64_t)e * p.sB) * S::E + (TRANS ? n0 * p.ldb : (int64_t)n0) * S::E;
    const char *A = p.A + (int64_t)r0 * p.lda * S::E;
    f32x4 acc[S::FRAGS];
#pragma unroll
    for (int j = 0; j < S::FRAGS; ++j) acc[j] = f32x4{0, 0, 0, 0};
    using Loads = StreamB<DT, TRANS>;
    auto fetch = [&](int s, Loads &b, StreamA<DT, TRANS> &a, auto part) {
        constexpr int PART = decltype(part)::value;
        const int k_left = p.K - s * S::K;
        b.template load<PART>(B + s * b_step, p.ldb, n_left, k_left, lane);
        a.template load<PART>(A + (int64_t)s * S::K * S::E, p.lda, rows, k_left, lane);
    };
    // whole stages, the next one's loads in flight during the current one's
    // products; then those that N or K cuts, one at a time
    const int whole = n_left < S::COLS || stages == 0 ? 0 : p.K / S::K;
    int s = wave;
    if (s < whole) {
        const std::integral_constant<int, Loads::ALL> full;
        StreamB<DT, TRANS> b0, b1;
        StreamA<DT, TRANS> a0, a1;
        fetch(s, b0, a0, full);
        for (;;) {
            s += waves;
            const bool more = s < whole;
            if (more) fetch(s, b1, a1, full);
            __builtin_amdgcn_sched_barrier(0);
            stream_mma<DT, TRANS>(b0, a0, acc);
            if (!more) break;
            b0 = b1;
            a0 = a1;
        }
    }
    const bool chunks = p.K % S::PER == 0 && (TRANS || p.N % S::PER == 0);
    for (; s < stages; s += waves) {
        StreamB<DT, TRANS> b;
        StreamA<DT, TRANS> a;
        // (25 rows, N 728, K 1912 transposed: 12.6 us element by element, 5.8 in chunks)
        if (chunks) fetch(s, b, a, std::integral_constant<int, Loads::CHUNKS>{});
        else fetch(s, b, a, std::integral_constant<int, Loads::ELEMENTS>{});
        stream_mma<DT, TRANS>(b, a, acc);
    }
#pragma unroll
    for (int j = 0; j < S::FRAGS; ++j) stream_lds[(wave * S::FRAGS + j) * 64 + lane] = acc[j];
    __syncthreads();
    // wave w sums and stores value w, w + waves, ... of the tile's four: the FRAGS
    // columns of a value are neighbours (B as stored), the four values of a
    // fragment are (B transposed)
    const int r = r0 + lane % 16, g = lane / 16;
    if constexpr (TRANS) {
        for (int j = wave; j < S::FRAGS; j += waves) {
            f32x4 v = stream_lds[j * 64 + lane];
            for (int w = 1; w < waves; ++w) v += stream_lds[(w * S::FRAGS + j) * 64 + lane];
            const int n = 16 * j + 4 * g;
            if (r < span.hi && n < n_left)
                store4<DT>(p.C, (int64_t)r * p.ldc + n0 + n, n_left - n, p.c_f32, wide, v);
        }
    } else {
        for (int q = wave; q < S::FRAGS; q += waves) {      // (value, four fragments)
            const int v = q / (S::FRAGS / 4), j0 = 4 * (q % (S::FRAGS / 4));
            f32x4 x;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float *at = reinterpret_cast<const float *>(stream_lds + (j0 + j) * 64 + lane) + v;
                float y = at[0];
                for (int w = 1; w < waves; ++w) y += at[w * S::FRAGS * 256];
                x[j] = y;
            }
            const int n = S::PER * (4 * g + v) + j0;
            if (r < span.hi && n < n_left)
                store4<DT>(p.C, (int64_t)r * p.ldc + n0 + n, n_left - n, p.c_f32, wide, x);
        }
    }
}

// C[g] = A[rows of g]^T . D[rows of g] where an extent is below kNarrow, of which a tile
// would be mostly empty: a thread a column of the longer extent and `width` of them a row,
// all of the shorter extent in its registers, an expert's rows dealt to the 1024 / width
// threads of a column, whose sums are added in LDS in their order.  Bound by the latency of
// the loads: 16384 rows, M 4096, N 4 bf16 341 us, M 7, N 7 38 us (with a thread an output
// and one running sum of an expert's rows 6240 and 1175).
constexpr int kNarrow = 8;
inline int narrow_width(int64_t longer, bool f32) {
    int w = 8;
    while (w < longer && w < (f32 ? 32 : 64)) w *= 2;      // a cache line of a row at most
    return w;
}
template <int DT>
__global__ __launch_bounds__(1024) void wgrad_narrow_kernel(GroupedParams p, int width) {
    typedef typename ElemOf<DT>::type T;
    __shared__ float part[(kNarrow - 1) * 1024];
    const bool m_short = p.M < p.N;
    const int few = m_short ? p.M : p.N, many = m_short ? p.N : p.M;
    const T *S = reinterpret_cast<const T *>(m_short ? p.A : p.B), *L = reinterpret_cast<const T *>(m_short ? p.B : p.A);
    const int64_t ld_s = m_short ? p.lda : p.ldb, ld_l = m_short ? p.ldb : p.lda;
    const int tid = threadIdx.x, slots = 1024 / width, x = blockIdx.x * width + tid % width, g = blockIdx.y;
    const RowSpan span = rows_of(p.offsets, g, p.experts, p.rows);
    float sum[kNarrow - 1] = {};
    int from[kNarrow - 1];          // past the extent its last again: loads without a branch, in flight together
#pragma unroll
    for (int j = 0; j < kNarrow - 1; ++j) from[j] = j < few ? j : few - 1;
    if (x < many) {
#pragma unroll 4
        for (int r = span.lo + tid / width; r < span.hi; r += slots) {
            const float v = (float)L[r * ld_l + x];
#pragma unroll
            for (int j = 0; j < kNarrow - 1; ++j) sum[j] = __builtin_fmaf(v, (float)S[r * ld_s + from[j]], sum[j]);
        }
    }
#pragma unroll
    for (int j = 0; j < kNarrow - 1; ++j)
        if (j < few) part[j * 1024 + tid] = sum[j];
    __syncthreads();
    for (int i = tid; i < few * width; i += 1024) {
        const int j = i / width, c = i % width, at = blockIdx.x * width + c;
        if (at >= many) continue;
        float v = part[j * 1024 + c];
        for (int k = 1; k < slots; ++k) v += part[j * 1024 + k * width + c];
        const int64_t to = (int64_t)g * p.sC + (m_short ? j * p.ldc + at : at * p.ldc + j);
        if (DT == DT_F32 || p.c_f32) reinterpret_cast<float *>(p.C)[to] = v;
        else reinterpret_cast<T *>(p.C)[to] = (T)v;
    }
}

}  // namespace tg
