// few_rows.hpp -- the gated pair, its gate's gradient, and a projection with adapters, for
// few rows: bound by the bytes of the weights, which are streamed from HBM to registers
// as grouped_stream.hpp does it (its stages, fragments and order of lanes).
//
// One matrix alone has few strips of columns, so K is split over workgroups too where
// that is needed to have all CUs load: each writes its fp32 sums to the caller's
// workspace, and a second kernel adds them in the order of the splits and applies what
// follows the product.  Measured (gated, bf16 and f16): 1 row of 2816 x 1024 transposed 7.4 us, of
// which the kernel is 5.3; 16 rows of 8192 x 4096 transposed 32 us (4.2 TB/s of weights).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gated.hpp"

namespace tg {

enum { PART_ALL = 0, PART_CHUNKS = 1, PART_ELEMENTS = 2 };       // StreamB's parts of a stage

// 16 bytes at p, of which `left` elements exist
template <int E, int PART>
__device__ __forceinline__ u32x4 load_part(const char *p, int left) {
    constexpr int PER = 16 / E;
    if (PART == PART_ALL || (PART == PART_CHUNKS && left > 0) || left >= PER)
        return *reinterpret_cast<const u32x4_unaligned *>(p);
    u32x4 v = {0u, 0u, 0u, 0u};
    if constexpr (PART == PART_ELEMENTS) {
#pragma unroll
        for (int e = 0; e < PER - 1; ++e) {
            if (e < left) {
                if constexpr (E == 4) v[e] = reinterpret_cast<const uint32_t *>(p)[e];
                else v[e / 2] |= (uint32_t)reinterpret_cast<const uint16_t *>(p)[e] << (16 * (e % 2));
            }
        }
    }
    return v;
}

// Rows of A by a pointer of this lane's own (its row of 16; NULL: none).
template <int DT, bool TRANS>
struct FewA : StreamA<DT, TRANS> {
    using S = StreamShape<DT, TRANS>;
    template <int PART>
    __device__ __forceinline__ void load(const char *row, int64_t k0, int k_left, int lane) {
        const int g = lane / 16;
#pragma unroll
        for (int s = 0; s < S::A_LOADS; ++s) {
            const int k = 4 * S::PER * s + S::PER * g;
            this->a[s] = u32x4{0u, 0u, 0u, 0u};
            if (row) this->a[s] = load_part<S::E, PART>(row + (k0 + k) * S::E, k_left - k);
        }
    }
};

// A strip of one matrix: StreamShape's columns.
template <int DT, bool TRANS>
struct OneStrip {
    using S = StreamShape<DT, TRANS>;
    static constexpr int COLS = S::COLS;
    const char *base;           // the strip's first element
    int64_t ld;
    int n_left;
    __device__ __forceinline__ int64_t step() const { return (TRANS ? (int64_t)S::K : S::K * ld) * S::E; }
    template <int PART>
    __device__ __forceinline__ void load(int s, int k_left, int lane, StreamB<DT, TRANS> &b) const {
        b.template load<PART>(base + s * step(), ld, n_left, k_left, lane);
    }
};

// The same columns, half as many, of two matrices: the fragments' lanes 0-7 of 16 (as
// stored), or their first fragment (transposed), are the first's.
template <int DT, bool TRANS>
struct TwoStrips {
    using S = StreamShape<DT, TRANS>;
    static constexpr int COLS = S::COLS / 2;
    const char *first, *second;
    const char *mine;            // as stored: this lane's matrix
    int64_t ld;
    int n_left;
    __device__ __forceinline__ TwoStrips(const char *a, const char *b, int64_t ld_, int left, int lane)
        : first(a), second(b), ld(ld_), n_left(left) {
        uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
        mine = reinterpret_cast<const char *>(lane % 16 < 8 ? x : y);
    }
    template <int PART>
    __device__ __forceinline__ void load(int s, int k_left, int lane, StreamB<DT, TRANS> &b) const {
        const int g = lane / 16, c = lane % 16;
        if constexpr (TRANS) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int k = 4 * S::PER * (i % 4) + S::PER * g;
                const int left = c < n_left ? k_left - k : 0;
                b.q[i] = load_part<S::E, PART>((i < 4 ? first : second) + (c * ld + (int64_t)s * S::K + k) * S::E, left);
            }
        } else {
            const int n = S::PER * (c % 8);
            const char *col = mine + n * S::E;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int k = DT == DT_F32 ? 16 * (i / 4) + 4 * g + i % 4 : 8 * g + i;
                const int left = k < k_left ? n_left - n : 0;
                b.q[i] = load_part<S::E, PART>(col + ((int64_t)s * S::K + k) * ld * S::E, left);
            }
        }
    }
};

// acc += the strip's columns times this wave's stages s, s + waves, ... below `end` of K
template <int DT, bool TRANS, class STRIP>
__device__ __forceinline__ void few_sum(const STRIP &strip, const char *row, int K, bool chunks, int s, int waves, int end,
                                        int lane, f32x4 (&acc)[StreamShape<DT, TRANS>::FRAGS]) {
    using S = StreamShape<DT, TRANS>;
    const int all = K / S::K, whole = strip.n_left < STRIP::COLS ? 0 : (all < end ? all : end);
    auto fetch = [&](int at, StreamB<DT, TRANS> &b, FewA<DT, TRANS> &a, auto part) {
        constexpr int PART = decltype(part)::value;
        const int k_left = K - at * S::K;
        strip.template load<PART>(at, k_left, lane, b);
        a.template load<PART>(row, (int64_t)at * S::K, k_left, lane);
    };
    // the next stage's loads in flight during the current one's products
    auto loop = [&](int last, auto part) {
        if (s >= last) return;
        StreamB<DT, TRANS> b0, b1;
        FewA<DT, TRANS> a0, a1;
        fetch(s, b0, a0, part);
        for (;;) {
            s += waves;
            const bool more = s < last;
            if (more) fetch(s, b1, a1, part);
            __builtin_amdgcn_sched_barrier(0);
            stream_mma<DT, TRANS>(b0, a0, acc);
            if (!more) break;
            b0 = b1;
            a0 = a1;
        }
    };
    if (strip.n_left >= STRIP::COLS) loop(whole, std::integral_constant<int, PART_ALL>{});
    else if (chunks) loop(end, std::integral_constant<int, PART_CHUNKS>{});
    for (; s < end; s += waves) {
        StreamB<DT, TRANS> b;
        FewA<DT, TRANS> a;
        if (chunks) fetch(s, b, a, std::integral_constant<int, PART_CHUNKS>{});
        else fetch(s, b, a, std::integral_constant<int, PART_ELEMENTS>{});
        stream_mma<DT, TRANS>(b, a, acc);
    }
}

// Four neighbouring columns of a row, summed over the waves' fragments in LDS, item `it`
// of S::FRAGS * 64 (OneStrip): row it's lane, n the first column.
template <int DT, bool TRANS>
__device__ __forceinline__ f32x4 few_item(const f32x4 *lds, int waves, int it, int &row, int &n) {
    using S = StreamShape<DT, TRANS>;
    const int lane = it % 64, q = it / 64, g = lane / 16;
    row = lane % 16;
    f32x4 x;
    if constexpr (TRANS) {
        n = 16 * q + 4 * g;
        x = lds[q * 64 + lane];
        for (int w = 1; w < waves; ++w) x += lds[(w * S::FRAGS + q) * 64 + lane];
    } else {
        const int v = q / (S::FRAGS / 4), j0 = 4 * (q % (S::FRAGS / 4));
        n = S::PER * (4 * g + v) + j0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float *at = reinterpret_cast<const float *>(lds + (j0 + j) * 64 + lane) + v;
            float y = at[0];
            for (int w = 1; w < waves; ++w) y += at[w * S::FRAGS * 256];
            x[j] = y;
        }
    }
    return x;
}

// ---- the gated pair -----------------------------------------------------------------
// grid: (strips x splits) x row tiles (row_slot)
template <int DT, bool TRANS>
__global__ __launch_bounds__(512) void gated_few_kernel(GatedParams p) {
    using S = StreamShape<DT, TRANS>;
    using Strips = TwoStrips<DT, TRANS>;
    extern __shared__ f32x4 stream_lds[];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int lane = threadIdx.x & 63, waves = blockDim.x >> 6;
    const int z = blockIdx.x % p.splits, n0 = blockIdx.x / p.splits * Strips::COLS;
    int e;
    RowSpan span;
    if (!row_slot<16>(p.offsets, p.experts, p.rows, slot_of(p.experts), e, span)) return;
    const bool dead = e == p.experts;
    const int r0 = span.lo, rows = span.hi - r0, stages = dead ? 0 : (p.K + S::K - 1) / S::K;
    const int64_t b = ((dead ? 0 : (int64_t)e * p.sB) + (TRANS ? n0 * p.ldb : (int64_t)n0)) * S::E;
    const Strips strips(p.B + b, p.Bu + b, p.ldb, p.N - n0, lane);
    const char *row = lane % 16 < rows ? p.A + (int64_t)(r0 + lane % 16) * p.lda * S::E : nullptr;
    f32x4 acc[S::FRAGS];
#pragma unroll
    for (int j = 0; j < S::FRAGS; ++j) acc[j] = f32x4{0, 0, 0, 0};
    int begin, end;
    split_range(stages, p.splits, z, begin, end);
    few_sum<DT, TRANS>(strips, row, p.K, p.K % S::PER == 0 && (TRANS || p.N % S::PER == 0), begin + wave, waves, end, lane,
                       acc);
#pragma unroll
    for (int j = 0; j < S::FRAGS; ++j) stream_lds[(wave * S::FRAGS + j) * 64 + lane] = acc[j];
    __syncthreads();
    const bool wide_h = wide_rows<DT>(p.C, p.ldc), wide_u = wide_rows<DT>(p.U, p.ldu) && wide_rows<DT>(p.V, p.ldu);
    constexpr int ITEMS = S::FRAGS * 32;
    for (int it = threadIdx.x; it < ITEMS; it += blockDim.x) {
        int m, n;
        f32x4 u, v;
        if constexpr (TRANS) {
            u = few_item<DT, TRANS>(stream_lds, waves, it, m, n);
            v = stream_lds[64 + it];
            for (int w = 1; w < waves; ++w) v += stream_lds[(w * S::FRAGS + 1) * 64 + it];
        } else {
            // lane groups 0 and 1 hold u, 2 and 3 the same columns of v
            const int at = it / 32 * 64 + it % 32;
            int again;
            v = few_item<DT, TRANS>(stream_lds, waves, at + 32, m, again);
            u = few_item<DT, TRANS>(stream_lds, waves, at, m, n);
        }
        const int left = p.N - n0 - n;
        if (m >= rows || left <= 0) continue;
        const int64_t r = r0 + m, c = n0 + n;
        if (p.splits > 1) {
            float *to = p.part + ((int64_t)z * 2 * p.rows + r) * p.N + c;
            const bool wide = p.N % 4 == 0;
            store4<DT_F32>(reinterpret_cast<char *>(to), 0, left, true, wide, u);
            store4<DT_F32>(reinterpret_cast<char *>(to), (int64_t)p.rows * p.N, left, true, wide, v);
            continue;
        }
        if (p.U) {
            store4<DT>(p.U, r * p.ldu + c, left, false, wide_u, u);
            store4<DT>(p.V, r * p.ldu + c, left, false, wide_u, v);
        }
        with_act(p.act, [&](auto a) {
            f32x4 h;
#pragma unroll
            for (int x = 0; x < 4; ++x) h[x] = gate_act<decltype(a)::value>(u[x]) * v[x];
            store4<DT>(p.C, r * p.ldc + c, left, false, wide_h, h);
        });
    }
}

// h, u and v from the splits' sums: a thread four neighbours of a row
template <int DT>
__global__ __launch_bounds__(256) void gated_join_kernel(GatedParams p) {
    const int64_t quads = (p.N + 3) / 4, at = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (at >= quads * p.rows) return;
    const int64_t r = at / quads, c = at % quads * 4, plane = (int64_t)p.rows * p.N;
    const int left = (int)(p.N - c);
    const bool wide = p.N % 4 == 0;
    const char *part = reinterpret_cast<const char *>(p.part);
    f32x4 u = {0, 0, 0, 0}, v = {0, 0, 0, 0};
    for (int z = 0; z < p.splits; ++z) {
        u += load4<DT_F32>(part, 2 * z * plane + r * p.N + c, left, wide);
        v += load4<DT_F32>(part, (2 * z + 1) * plane + r * p.N + c, left, wide);
    }
    if (p.U) {
        const bool wide_u = wide_rows<DT>(p.U, p.ldu) && wide_rows<DT>(p.V, p.ldu);
        store4<DT>(p.U, r * p.ldu + c, left, false, wide_u, u);
        store4<DT>(p.V, r * p.ldu + c, left, false, wide_u, v);
    }
    with_act(p.act, [&](auto a) {
        f32x4 h;
#pragma unroll
        for (int x = 0; x < 4; ++x) h[x] = gate_act<decltype(a)::value>(u[x]) * v[x];
        store4<DT>(p.C, r * p.ldc + c, left, false, wide_rows<DT>(p.C, p.ldc), h);
    });
}

// The gate's gradient; K is split over the waves alone (plan_gate_grad_as).
template <int DT, bool TRANS>
__global__ __launch_bounds__(512) void gate_grad_few_kernel(GatedParams p) {
    using S = StreamShape<DT, TRANS>;
    extern __shared__ f32x4 stream_lds[];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int lane = threadIdx.x & 63, waves = blockDim.x >> 6, n0 = blockIdx.x * S::COLS;
    int e;
    RowSpan span;
    if (!row_slot<16>(p.offsets, p.experts, p.rows, slot_of(p.experts), e, span)) return;
    const bool dead = e == p.experts;
    const int r0 = span.lo, rows = span.hi - r0, stages = dead ? 0 : (p.K + S::K - 1) / S::K;
    const OneStrip<DT, TRANS> strip = {
        p.B + ((dead ? 0 : (int64_t)e * p.sB) + (TRANS ? n0 * p.ldb : (int64_t)n0)) * S::E, p.ldb, p.N - n0};
    const char *row = lane % 16 < rows ? p.A + (int64_t)(r0 + lane % 16) * p.lda * S::E : nullptr;
    f32x4 acc[S::FRAGS];
#pragma unroll
    for (int j = 0; j < S::FRAGS; ++j) acc[j] = f32x4{0, 0, 0, 0};
    few_sum<DT, TRANS>(strip, row, p.K, p.K % S::PER == 0 && (TRANS || p.N % S::PER == 0), wave, waves, stages, lane, acc);
#pragma unroll
    for (int j = 0; j < S::FRAGS; ++j) stream_lds[(wave * S::FRAGS + j) * 64 + lane] = acc[j];
    __syncthreads();
    const GateGrad how = gate_grad_of<DT>(p, dead);
    for (int it = threadIdx.x; it < S::FRAGS * 64; it += blockDim.x) {
        int m, n;
        const f32x4 dh = few_item<DT, TRANS>(stream_lds, waves, it, m, n);
        const int left = p.N - n0 - n;
        if (m < rows && left > 0)
            with_act(p.act, [&](auto a) { gate_grad4<DT, decltype(a)::value>(p, how, r0 + m, n0 + n, left, dh); });
    }
}

}  // namespace tg
