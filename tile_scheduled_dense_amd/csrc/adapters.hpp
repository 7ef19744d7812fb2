// adapters.hpp -- a projection shared by all rows with a low-rank adapter of each row's
// own beside it, and the adapters' gradients:
//
//   t[r] = scales[g] * (x[r] . A[g]),   y[r] = x[r] . W + t[r] . B[g]
//   d_A[g] = x^T . d_t,   d_B[g] = t^T . d_y        over the rows r of adapter g
//
// Position p of the adapters' order is row order[p] of x, y and t (order NULL: row p);
// adapter g has the positions offsets[g] .. offsets[g + 1], and those behind the last
// adapter's have none.
//
//  * Few rows (the bytes of W; adapters_few): one launch sums x . W (K split over workgroups) and
//    x . A[g] (16 positions of one adapter a workgroup, K split) into fp32 partial sums, a
//    second one adds them and t . B[g] position by position.
//  * More rows: t first (64 positions of one adapter a workgroup, K split, then added up and
//    rounded once to the inputs' type: it is the second product's operand), then the
//    block tiles of grouped_ring.hpp over positions, whose contraction goes on through
//    t and the B[g] of every adapter that has positions in the tile, the others' rows of t
//    being zeros.  Tiles that mix adapters keep W's product as dense as without any.
//  * Gradients: products whose contraction is an adapter's rows, the wide operand
//    straight from memory to registers, the narrow one transposed in LDS; a workgroup takes a
//    chunk of an adapter's rows, a second launch adds the chunks in their order.
//
// Measured, inputs that change from call to call: 1 row, rank 16, 4096 x 4096 bf16 12.9 us
// (33.8 MB; under a profiler the sums 10.7, the join 3.8); 64 rows of 20 adapters of rank 32
// 16.7 us (12 and 5.6); 8192 rows, 4 adapters of rank 64, 4096 x 4096 f16 252 us, of which t is 28
// (x from HBM while the last results go there) and the product 222 (1270 TFLOP/s); gradients of two
// adapters of rank 16, 8192 rows of 2048 and 4096, 27 us (100 MB, 3.7 TB/s) and 6 to add up.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "few_rows.hpp"
#include "narrow.hpp"

namespace tg {

struct AdapterParams : GroupedParams {   // A: x, B: W, C: y; experts: adapters; sB unused
    const char *down, *up;                // the adapters' A and B
    const float *scales;                  // NULL: 1
    const int32_t *order;
    char *T;                              // NULL: not stored
    char *low;                            // many rows: t of dtype by position, rows of ld_low
    float *part, *part_t;                 // fp32 sums by split of K: of x . W by row, of x . A[g] by position
    int64_t ld_down, s_down, ld_up, s_up, ldt;
    int64_t ld_low;
    int rank, splits, t_splits;
};

// The adapter of position p: the last of the groups 0 .. adapters (the last: none) that
// starts at or before it.  The same p in the whole wave.
__device__ __forceinline__ int group_of(const int32_t *offsets, int adapters, int p) {
    const int lane = threadIdx.x & 63, groups = adapters + 1, run = (groups + 63) / 64;
    int base = 0;
    if (run > 1) {
        const int i = lane * run;
        const uint64_t m = __ballot(i < groups && offsets[i < groups ? i : 0] <= p);
        base = m ? (63 - __builtin_clzll(m)) * run : 0;
    }
    const int i = base + lane;
    const uint64_t m = __ballot(i < groups && (run == 1 || lane < run) && offsets[i < groups ? i : 0] <= p);
    return m ? base + 63 - __builtin_clzll(m) : base;
}

__device__ __forceinline__ int row_at(const AdapterParams &p, int pos) {
    return p.order ? row_in(p.order, pos, p.rows) : pos;
}

// ---- x . A[g] -----------------------------------------------------------------------------
// 16 positions of one adapter, COLS of its rank, the stages of one split: sums into LDS.
// false: no such positions.
template <int DT, bool TRANS>
__device__ __forceinline__ bool shrink_sum(const AdapterParams &p, int strip, int slot, int split, f32x4 *lds, int &g,
                                           RowSpan &span) {
    using S = StreamShape<DT, TRANS>;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int lane = threadIdx.x & 63, waves = blockDim.x >> 6, n0 = strip * S::COLS;
    if (!row_slot<16>(p.offsets, p.experts, p.rows, slot, g, span)) return false;
    const bool dead = g == p.experts;
    const int rows = span.hi - span.lo, stages = dead ? 0 : (p.K + S::K - 1) / S::K;
    const OneStrip<DT, TRANS> of = {
        p.down + ((dead ? 0 : (int64_t)g * p.s_down) + (TRANS ? n0 * p.ld_down : (int64_t)n0)) * S::E, p.ld_down,
        p.rank - n0};
    const char *row =
        lane % 16 < rows ? p.A + (int64_t)row_at(p, span.lo + lane % 16) * p.lda * S::E : nullptr;
    f32x4 acc[S::FRAGS];
#pragma unroll
    for (int j = 0; j < S::FRAGS; ++j) acc[j] = f32x4{0, 0, 0, 0};
    int begin, end;
    split_range(stages, p.t_splits, split, begin, end);
    few_sum<DT, TRANS>(of, row, p.K, p.K % S::PER == 0 && (TRANS || p.rank % S::PER == 0), begin + wave, waves, end, lane,
                       acc);
#pragma unroll
    for (int j = 0; j < S::FRAGS; ++j) lds[(wave * S::FRAGS + j) * 64 + lane] = acc[j];
    __syncthreads();
    return true;
}

// The sums of shrink_sum by split and position (few rows).
template <int DT, bool TRANS>
__device__ __forceinline__ void shrink_few(const AdapterParams &p, int id, int strips, f32x4 *lds) {
    using S = StreamShape<DT, TRANS>;
    const int split = id % p.t_splits, strip = id / p.t_splits % strips, slot = id / p.t_splits / strips;
    const int waves = blockDim.x >> 6, n0 = strip * S::COLS;
    int g;
    RowSpan span;
    if (!shrink_sum<DT, TRANS>(p, strip, slot - (p.experts + 1), split, lds, g, span) || g == p.experts) return;
    for (int it = threadIdx.x; it < S::FRAGS * 64; it += blockDim.x) {
        int m, n;
        const f32x4 v = few_item<DT, TRANS>(lds, waves, it, m, n);
        const int left = p.rank - n0 - n;
        if (m < span.hi - span.lo && left > 0)
            store4<DT_F32>(reinterpret_cast<char *>(p.part_t), ((int64_t)split * p.rows + span.lo + m) * p.rank + n0 + n,
                           left, true, p.rank % 4 == 0, v);
    }
}

// ---- few rows -------------------------------------------------------------------------------
// Workgroups below `low`: x . A[g] (they are the longer chains, so they start first); behind
// them x . W, strips x splits x tiles of 16 rows.
template <int DT, bool TRANS>
__global__ __launch_bounds__(512) void adapters_few_kernel(AdapterParams p, int low, int row_tiles, int strips_t) {
    using S = StreamShape<DT, TRANS>;
    extern __shared__ f32x4 stream_lds[];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int lane = threadIdx.x & 63, waves = blockDim.x >> 6;
    int id = blockIdx.x;
    if (id < low) {
        shrink_few<DT, TRANS>(p, id, strips_t, stream_lds);
        return;
    }
    id -= low;
    const int z = id % p.splits, tile = id / p.splits % row_tiles, n0 = id / p.splits / row_tiles * S::COLS;
    const int r0 = 16 * tile, stages = (p.K + S::K - 1) / S::K;
    const OneStrip<DT, TRANS> of = {p.B + (TRANS ? n0 * p.ldb : (int64_t)n0) * S::E, p.ldb, p.N - n0};
    const char *row = r0 + lane % 16 < p.rows ? p.A + (int64_t)(r0 + lane % 16) * p.lda * S::E : nullptr;
    f32x4 acc[S::FRAGS];
#pragma unroll
    for (int j = 0; j < S::FRAGS; ++j) acc[j] = f32x4{0, 0, 0, 0};
    int begin, end;
    split_range(stages, p.splits, z, begin, end);
    few_sum<DT, TRANS>(of, row, p.K, p.K % S::PER == 0 && (TRANS || p.N % S::PER == 0), begin + wave, waves, end, lane, acc);
#pragma unroll
    for (int j = 0; j < S::FRAGS; ++j) stream_lds[(wave * S::FRAGS + j) * 64 + lane] = acc[j];
    __syncthreads();
    for (int it = threadIdx.x; it < S::FRAGS * 64; it += blockDim.x) {
        int m, n;
        const f32x4 v = few_item<DT, TRANS>(stream_lds, waves, it, m, n);
        const int left = p.N - n0 - n;
        if (r0 + m < p.rows && left > 0)
            store4<DT_F32>(reinterpret_cast<char *>(p.part), ((int64_t)z * p.rows + r0 + m) * p.N + n0 + n, left, true,
                           p.N % 4 == 0, v);
    }
}

// The same where W is read in tiles of BM rows through LDS.
template <class C, bool KS, int STAGES>
__global__ __launch_bounds__(C::THREADS, C::OCCUPANCY) void adapters_split_kernel(AdapterParams p, int low, int strips_t) {
    using S = StreamShape<C::DT, !KS>;
    constexpr int TILE = GroupedTile<C, false, KS, STAGES>::LDS, SUMS = C::WAVES * S::FRAGS * 1024;
    __shared__ __attribute__((aligned(1024))) char smem[TILE > SUMS ? TILE : SUMS];
    int id = blockIdx.x;
    if (id < low) {
        shrink_few<C::DT, !KS>(p, id, strips_t, reinterpret_cast<f32x4 *>(smem));
        return;
    }
    id -= low;
    const int strips = (p.N + C::BN - 1) / C::BN;
    const int z = id % p.splits, n0 = id / p.splits % strips * C::BN, m0 = id / p.splits / strips * C::BM;
    int begin, end;
    split_range((p.K + C::BK - 1) / C::BK, p.splits, z, begin, end);
    const int k0 = begin * C::BK, K = (end * C::BK < p.K ? end * C::BK : p.K) - k0;
    GroupedTile<C, false, KS, STAGES> tile;
    tile.init(p.A + ((int64_t)m0 * p.lda + k0) * C::ELEM, p.lda, p.rows - m0,
              p.B + (KS ? k0 * p.ldb + n0 : n0 * p.ldb + k0) * C::ELEM, p.ldb, p.N - n0, K > 0 ? K : 0, smem);
    tile.run_ring();
    tile.store(reinterpret_cast<char *>(p.part), ((int64_t)z * p.rows + m0) * p.N + n0, p.N, p.rows - m0, p.N - n0, true,
               false);
}

// y and t of a position from the sums (workgroups: position by position): y's sums over the
// splits, t's in fp32 through LDS, kJoinRank of the rank at a time.  A thread has COLS
// neighbouring columns: two of B's rows as stored, one of its columns transposed (whose
// rank is contiguous); the next STEP ranks' loads of B are in flight, the first before t
// is there.  (As stored with four columns and eight ranks at a time: 64 rows of rank 32, 4096
// columns, 14 us.)
constexpr int kJoinRank = 256;
template <bool TRANS> constexpr int join_cols() { return TRANS ? 1 : 2; }
// workgroups of a position; one without columns too, for T
template <bool TRANS>
__host__ __device__ constexpr int64_t join_parts(int64_t N) {
    return N > 0 ? (N + 256 * join_cols<TRANS>() - 1) / (256 * join_cols<TRANS>()) : 1;
}
template <int DT, bool TRANS>
__global__ __launch_bounds__(256) void adapters_join_kernel(AdapterParams p) {
    typedef typename ElemOf<DT>::type E;
    typedef E Two __attribute__((ext_vector_type(2)));
    typedef Two __attribute__((aligned(sizeof(E)))) TwoAnywhere;
    constexpr int COLS = join_cols<TRANS>(), STEP = TRANS ? Chunk<DT>::PER : 16, BYTES = (int)sizeof(E);
    __shared__ float t[kJoinRank + STEP];
    const int parts = (int)join_parts<TRANS>(p.N), pos = blockIdx.x / parts, part = blockIdx.x % parts;
    const int g = group_of(p.offsets, p.experts, pos);
    const int64_t r = row_at(p, pos);
    const int c = COLS * (part * 256 + (int)threadIdx.x), left = p.N - c;
    const bool has = g < p.experts;
    const char *up = p.up + (has ? (int64_t)g * p.s_up : 0) * BYTES;
    // B of ranks k .. k + STEP - 1
    struct Piece {
        Two rows[TRANS ? 1 : STEP];
        Chunk<DT> column;
    };
    auto fetch = [&](int k, Piece &b) {
        if constexpr (TRANS) {
            b.column.load(up, (int64_t)c * p.ld_up + k, has && left > 0 ? p.rank - k : 0);
        } else {
            const E *at = reinterpret_cast<const E *>(up) + (int64_t)k * p.ld_up + c;
#pragma unroll
            for (int i = 0; i < STEP; ++i) {
                b.rows[i] = Two{};
                if (has && k + i < p.rank) {
                    if (left >= 2) b.rows[i] = *reinterpret_cast<const TwoAnywhere *>(at);
                    else if (left == 1) b.rows[i][0] = at[0];
                }
                at += p.ld_up;
            }
        }
    };
    Piece b0, b1;
    fetch(0, b0);
    float y[COLS] = {};
    if (left > 0) {
        const float *sums = p.part + r * p.N + c;
        const int64_t plane = (int64_t)p.rows * p.N;
#pragma unroll 4
        for (int z = 0; z < p.splits; ++z) {
            y[0] += sums[z * plane];
            if (COLS > 1 && left > 1) y[COLS - 1] += sums[z * plane + 1];
        }
    }
    const float scale = has ? (p.scales ? p.scales[g] : 1.0f) : 0.0f;
    for (int base = 0; base < p.rank; base += kJoinRank) {
        const int n = p.rank - base < kJoinRank ? p.rank - base : kJoinRank;
        if (base) __syncthreads();
        for (int k = threadIdx.x; k < kJoinRank + STEP; k += 256) {
            float s = 0;
            if (has && k < n) {
                const float *sums = p.part_t + (int64_t)pos * p.rank + base + k;
#pragma unroll 8
                for (int z = 0; z < p.t_splits; ++z) s += sums[(int64_t)z * p.rows * p.rank];
                s *= scale;
            }
            t[k] = s;
            if (p.T && part == 0 && k < n) reinterpret_cast<E *>(p.T)[r * p.ldt + base + k] = (E)s;
        }
        __syncthreads();
        if (!has) continue;
        for (int k = 0; k < n; k += STEP) {
            if (base + k + STEP < p.rank) fetch(base + k + STEP, b1);
#pragma unroll
            for (int i = 0; i < STEP; ++i) {
                if constexpr (TRANS) {
                    y[0] = __builtin_fmaf(t[k + i], (float)b0.column.x[i], y[0]);
                } else {
#pragma unroll
                    for (int e = 0; e < COLS; ++e) y[e] = __builtin_fmaf(t[k + i], (float)b0.rows[i][e], y[e]);
                }
            }
            b0 = b1;
        }
    }
    E *to = reinterpret_cast<E *>(p.C) + r * p.ldc + c;
    if (left >= COLS) {
        if constexpr (TRANS) to[0] = (E)y[0];
        else *reinterpret_cast<TwoAnywhere *>(to) = Two{(E)y[0], (E)y[1]};
    } else if (left > 0) {
        to[0] = (E)y[0];
    }
}

// ---- many rows ------------------------------------------------------------------------------
// A's operand whose rows lie at order[m]: offsets from the matrix's first element.
template <class V, int T>
struct OrderedOperand : RingOperand<V, false, T> {
    using O = RingOperand<V, false, T>;
    int at[O::PER];
    // base_: the matrix; order: of the tile's first row
    __device__ __forceinline__ void init(const char *base_, int64_t ld_, int left_, int w, uint32_t lds_, int lane_,
                                         int wave_, const int32_t *order, int total) {
        O::init(base_, ld_, left_, w, lds_, lane_, wave_);
#pragma unroll
        for (int d = 0; d < O::PER; ++d) {
            at[d] = this->x[d] < left_ ? row_in(order, this->x[d], total) * (int)ld_ : 0;
            const int off = this->x[d] < left_ ? (at[d] + this->k[d]) * O::E : kOutOfRange;
            this->voff[d] = off + O::SHIFT - 1024 * O::CP::pos(d);
        }
    }
    __device__ __forceinline__ void tail_load(int64_t k0, int K, u32x4 *tail) const {
        const rsrc_t r = make_rsrc(this->base + k0 * O::E);
#pragma unroll
        for (int d = 0; d < O::PER; ++d) {
            const int run = K - (int)k0 - this->k[d];
            const int n = this->x[d] >= this->left || run <= 0 ? 0 : (run < O::CHUNK ? run : O::CHUNK);
            tail[d] = bload16_n<O::E>(r, n > 0 ? (at[d] + this->k[d]) * O::E : 0, 0, n);
        }
    }
};

// x's rows at positions m0 .. , in order or through the table
template <class C, bool ORDERED>
using OperandX = typename std::conditional<ORDERED, OrderedOperand<C, C::TM>, OperandA<C, false>>::type;

template <class C, bool KS, bool ORDERED, int STAGES>
struct AdapterTile : GroupedTile<C, false, KS, STAGES, OperandX<C, ORDERED>, OperandB<C, KS>> {
    using OA = OperandX<C, ORDERED>;
    using OB = OperandB<C, KS>;

    // positions m0 .. of which m_left exist, from k0 on K of them; B: the second operand's
    // first element
    __device__ __forceinline__ void init(const AdapterParams &p, int m0, int m_left, int k0, int K, const char *B, int64_t ldb,
                                         int n_left, char *smem) {
        this->begin(K, !KS || n_left >= C::BN || n_left % C::CHUNK == 0);
        const uint32_t lds0 = lds_address(smem);
        this->b.init(B, ldb, n_left, (this->wave % C::WAVES_N) * C::WTN, lds0, this->lane, this->wave);
        const int w = (this->wave / C::WAVES_N) * C::WTM;
        const char *A = p.A + (int64_t)k0 * C::ELEM;
        if constexpr (ORDERED)
            this->a.init(A, p.lda, m_left, w, lds0 + STAGES * OB::REGION, this->lane, this->wave, p.order + m0, p.rows);
        else
            this->a.init(A + (int64_t)m0 * p.lda * C::ELEM, p.lda, m_left, w, lds0 + STAGES * OB::REGION, this->lane,
                         this->wave);
        this->acc.zero();
    }

    // f(g, lo, hi) for every adapter with positions in the tile: lo .. hi, from its first
    template <class F>
    __device__ __forceinline__ static void each_adapter(const AdapterParams &p, int m0, const F &f) {
        const int lane = threadIdx.x & 63, m_end = m0 + C::BM < p.rows ? m0 + C::BM : p.rows;
        const int last = group_of(p.offsets, p.experts, m_end - 1);
        for (int base = group_of(p.offsets, p.experts, m0); base <= last; base += 64) {
            const int g = base + lane;
            RowSpan s = {0, 0};
            if (g <= last && g < p.experts) s = rows_of(p.offsets, g, p.experts, p.rows);
            const int lo = s.lo > m0 ? s.lo - m0 : 0, hi = (s.hi < m_end ? s.hi : m_end) - m0;
            for (uint64_t m = __ballot(lo < hi); m; m &= m - 1) {
                const int l = __builtin_ctzll(m);
                f(base + l, __builtin_amdgcn_readlane(lo, l), __builtin_amdgcn_readlane(hi, l));
            }
        }
    }

    // A K tile from registers through the first LDS copy, whose last readers are done.
    __device__ __forceinline__ void multiply(const u32x4 (&ta)[OA::PER], const u32x4 (&tb)[OB::PER]) {
        this->a.tail_store(0, ta);
        this->b.tail_store(0, tb);
        wait_lds();
        block_barrier();
        u32x4 fa[C::TM], fb[C::TN];
#pragma unroll
        for (int r = 0; r < AdapterTile::READS; ++r) this->read_piece(0, r, fa, fb);
        static_for<0, AdapterTile::NMFMA, 1>([&](auto q) { this->template mma<false, decltype(q)::value>(fa, fb); });
        wait_lds();
    }
    // The K tile at k0, behind those of the ring, of K in all.
    __device__ __forceinline__ void cut_tile(int k0, int K) {
        u32x4 ta[OA::PER], tb[OB::PER];
        this->a.tail_load(k0, K, ta);
        this->b.tail_load(k0, K, tb);
        block_barrier();
        multiply(ta, tb);
        this->acc.settle();
    }

    // The K tile of B[g] at rank k0 (columns from n0), zeros past its ends; whether any of
    // the workgroup's values is not finite.
    __device__ __forceinline__ void load_up(const AdapterParams &p, int g, int n0, int k0, u32x4 (&tb)[OB::PER]) const {
        const char *up = p.up + ((int64_t)g * p.s_up + (KS ? k0 * p.ld_up + n0 : n0 * p.ld_up + k0)) * C::ELEM;
        const rsrc_t rb = make_rsrc(up);
#pragma unroll
        for (int d = 0; d < OB::PER; ++d) {
            const int k_left = p.rank - k0 - this->b.k[d], x_left = this->b.left - this->b.x[d];
            const int run = KS ? x_left : k_left, other = KS ? k_left : x_left;
            const int n = other <= 0 || run <= 0 ? 0 : (run < C::CHUNK ? run : C::CHUNK);
            const int at = KS ? this->b.k[d] * (int)p.ld_up + this->b.x[d] : this->b.x[d] * (int)p.ld_up + this->b.k[d];
            tb[d] = bload16_n<C::ELEM>(rb, n > 0 ? at * C::ELEM : 0, 0, n);
        }
    }
    static constexpr uint32_t EXP = C::DT == DT_F32 ? 0x7f800000u : (C::DT == DT_BF16 ? 0x7f80u : 0x7c00u);
    __device__ __forceinline__ static bool not_finite(const u32x4 (&t)[OB::PER]) {
        bool bad = false;
#pragma unroll
        for (int d = 0; d < OB::PER; ++d)
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                bad |= (t[d][w] & EXP) == EXP;
                if (C::DT != DT_F32) bad |= (t[d][w] >> 16 & EXP) == EXP;
            }
        return __syncthreads_or(bad);
    }
    // the values that are not finite as zeros
    __device__ __forceinline__ static void clear_not_finite(u32x4 (&t)[OB::PER]) {
#pragma unroll
        for (int d = 0; d < OB::PER; ++d)
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                uint32_t x = t[d][w];
                if (C::DT == DT_F32) {
                    x = (x & EXP) == EXP ? 0 : x;
                } else {
                    x = (x & EXP) == EXP ? x & 0xffff0000u : x;
                    x = (x >> 16 & EXP) == EXP ? x & 0xffffu : x;
                }
                t[d][w] = x;
            }
    }

    // The contraction goes on: t . B[g] for every adapter with positions in the tile, in
    // K tiles of the rank through registers, one at a time (an adapter of 32 and less is
    // one), other adapters' rows and what lies past the rank as zeros.  Those zeros would make
    // NaN of an infinity or NaN in B[g], in other adapters' rows: such values are left out,
    // and true is returned, unless all of the tile's positions are g's.
    __device__ __forceinline__ bool adapters(const AdapterParams &p, int m0, int n0) {
        const int m_here = p.rows - m0 < C::BM ? p.rows - m0 : C::BM;
        const rsrc_t rt = make_rsrc(p.low + (int64_t)m0 * p.ld_low * C::ELEM);
        bool left_out = false;
        each_adapter(p, m0, [&](int g, int lo, int hi) {
            for (int k0 = 0; k0 < p.rank; k0 += C::BK) {
                u32x4 ta[OA::PER], tb[OB::PER];
#pragma unroll
                for (int d = 0; d < OA::PER; ++d) {
                    const int x = this->a.x[d], k = k0 + this->a.k[d];
                    const bool in = x >= lo && x < hi && k < p.ld_low;
                    ta[d] = bload16(rt, in ? (x * (int)p.ld_low + k) * C::ELEM : kOutOfRange, 0);
                }
                load_up(p, g, n0, k0, tb);
                if (hi - lo < m_here) {
                    if (not_finite(tb)) {
                        left_out = true;
                        clear_not_finite(tb);
                    }
                } else {
                    block_barrier();               // the copy's last readers are done
                }
                multiply(ta, tb);
            }
        });
        this->acc.settle();
        return left_out;
    }
    // What adapters() left out, element by element, onto the stored result: add(position in
    // the tile, column, sum).  Such a sum is an infinity or NaN, so that the result's rounding
    // does not matter (but an infinity that it made of a large value counts as one).
    template <class F>
    __device__ __forceinline__ void left_out(const AdapterParams &p, int m0, int n0, const F &add) const {
        typedef typename ElemOf<C::DT>::type T;
        const int n_here = p.N - n0 < C::BN ? p.N - n0 : C::BN, m_here = p.rows - m0 < C::BM ? p.rows - m0 : C::BM;
        __threadfence_block();
        __syncthreads();
        each_adapter(p, m0, [&](int g, int lo, int hi) {
            if (hi - lo == m_here) return;
            const T *up = reinterpret_cast<const T *>(p.up) + (int64_t)g * p.s_up;
            const T *low = reinterpret_cast<const T *>(p.low) + (int64_t)m0 * p.ld_low;
            for (int k0 = 0; k0 < p.rank; k0 += C::BK) {
                u32x4 tb[OB::PER];
                load_up(p, g, n0, k0, tb);
                if (!not_finite(tb)) continue;
                const int k_end = k0 + C::BK < p.rank ? k0 + C::BK : p.rank;
                for (int i = threadIdx.x; i < (hi - lo) * n_here; i += C::THREADS) {
                    const int m = lo + i / n_here, n = i % n_here;
                    float sum = 0;
                    bool any = false;
                    for (int k = k0; k < k_end; ++k) {
                        const float b = (float)(KS ? up[k * p.ld_up + n0 + n] : up[(n0 + n) * p.ld_up + k]);
                        if (__builtin_isfinite(b)) continue;
                        sum += (float)low[m * p.ld_low + k] * b;
                        any = true;
                    }
                    if (any) add(m, n, sum);
                }
            }
        });
    }
    __device__ __forceinline__ void store_rows(const AdapterParams &p, int m0, int n0) const {
        const auto value = [&](auto i, auto j, auto v) {
            return this->acc.get(decltype(i)::value, decltype(j)::value, decltype(v)::value);
        };
        if constexpr (ORDERED)
            TileStore<C, C::TN, decltype(value), true>{value, this->lane, this->wave, p.order + m0, p.rows}.store(
                p.C, n0, p.ldc, p.rows - m0, p.N - n0, false, p.past);
        else
            TileStore<C, C::TN, decltype(value)>{value, this->lane, this->wave}.store(
                p.C, (int64_t)m0 * p.ldc + n0, p.ldc, p.rows - m0, p.N - n0, false, p.past);
    }
};

// x . A[g] of up to 64 positions of one adapter, 64 of the rank and a split of K, times the
// adapter's scale, into part_t.  grid: (rank x splits) x row tiles.
template <class C, bool KS, bool ORDERED, int STAGES>
__global__ __launch_bounds__(C::THREADS, C::OCCUPANCY) void shrink_tile_kernel(AdapterParams p) {
    __shared__ __attribute__((aligned(1024))) char smem[AdapterTile<C, KS, ORDERED, STAGES>::LDS];
    const int z = blockIdx.x % p.t_splits, n0 = (int)(blockIdx.x / p.t_splits) * C::BN;
    int g;
    RowSpan span;
    if (!row_slot<C::BM>(p.offsets, p.experts, p.rows, slot_of(p.experts), g, span)) return;
    const bool has = g < p.experts;
    int begin = 0, end = 0;
    if (has) split_range((p.K + C::BK - 1) / C::BK, p.t_splits, z, begin, end);
    const int k0 = begin * C::BK, K = (end * C::BK < p.K ? end * C::BK : p.K) - k0, rows = span.hi - span.lo;
    const char *B = p.down + ((has ? (int64_t)g * p.s_down : 0) + (KS ? k0 * p.ld_down + n0 : n0 * p.ld_down + k0)) * C::ELEM;
    const int ring = KS ? ring_rows(K > 0 ? K : 0, p.rank, C::BK, C::CHUNK) : (K > 0 ? K : 0);
    AdapterTile<C, KS, ORDERED, STAGES> tile;
    tile.init(p, span.lo, rows, k0, ring, B, p.ld_down, p.rank - n0, smem);
    tile.run_ring();
    if (KS && ring < K) tile.cut_tile(ring, K);
    const float scale = has && p.scales ? p.scales[g] : 1.0f;
    const auto value = [&](auto i, auto j, auto v) {
        return tile.acc.get(decltype(i)::value, decltype(j)::value, decltype(v)::value) * scale;
    };
    TileStore<C, C::TN, decltype(value)>{value, tile.lane, tile.wave}.store(
        reinterpret_cast<char *>(p.part_t), ((int64_t)z * p.rows + span.lo) * p.rank + n0, p.rank, rows, p.rank - n0, true,
        false);
}

// t of dtype from the splits' sums, into low (its rows' rest up to ld_low zeros) and T: a
// thread four neighbours.  t is rounded once: it is the next product's operand.
template <int DT>
__global__ __launch_bounds__(256) void shrink_join_kernel(AdapterParams p) {
    const int quads = (int)p.ld_low / 4;
    const int64_t at = (int64_t)blockIdx.x * 256 + threadIdx.x, plane = (int64_t)p.rows * p.rank;
    if (at >= (int64_t)p.rows * quads) return;
    const int pos = (int)(at / quads), k = (int)(at % quads) * 4, left = p.rank - k;
    f32x4 v = {0, 0, 0, 0};
#pragma unroll 4
    for (int z = 0; z < p.t_splits; ++z)
        v += load4<DT_F32>(reinterpret_cast<const char *>(p.part_t), z * plane + (int64_t)pos * p.rank + k, left,
                           p.rank % 4 == 0);
    store4<DT>(p.low, (int64_t)pos * p.ld_low + k, 4, false, true, v);
    if (p.T && left > 0) store4<DT>(p.T, (int64_t)row_at(p, pos) * p.ldt + k, left, false, wide_rows<DT>(p.T, p.ldt), v);
}

template <class C, bool KS, bool ORDERED, bool PIPE, int STAGES>
__device__ __forceinline__ void run_adapters(const AdapterParams &p, char *smem, int m0, int n0) {
    typedef typename ElemOf<C::DT>::type T;
    AdapterTile<C, KS, ORDERED, STAGES> tile;
    tile.init(p, m0, p.rows - m0, 0, p.K, p.B + (KS ? (int64_t)n0 : n0 * p.ldb) * C::ELEM, p.ldb, p.N - n0, smem);
    if constexpr (PIPE) tile.run_pipe();
    else tile.run_ring();
    const bool more = tile.adapters(p, m0, n0);
    tile.store_rows(p, m0, n0);
    if (more)
        tile.left_out(p, m0, n0, [&](int m, int n, float sum) {
            T *y = reinterpret_cast<T *>(p.C) + (int64_t)(ORDERED ? row_in(p.order, m0 + m, p.rows) : m0 + m) * p.ldc + n0 + n;
            *y = (T)((float)*y + sum);
        });
}

// Tiles over positions, whatever their adapters; P: the pieces' configuration (C: none).
template <class C, class P, bool KS, bool ORDERED, bool PIPE, int STAGES>
__global__ __launch_bounds__(C::THREADS, C::OCCUPANCY) void adapters_tile_kernel(AdapterParams p) {
    constexpr bool PIECES = !std::is_same<C, P>::value;
    __shared__ __attribute__((aligned(1024))) char smem[AdapterTile<C, KS, ORDERED, STAGES>::LDS];
    GroupedParams whole = p;
    whole.offsets = nullptr;
    whole.experts = 1;
    RowTile t;
    if (!row_tile<C::BM, C::BN, PIECES>(whole, t)) return;
    if (PIECES && t.piece) run_adapters<P, KS, ORDERED, PIPE, STAGES>(p, smem, t.m0, t.n0);
    else run_adapters<C, KS, ORDERED, PIPE, STAGES>(p, smem, t.m0, t.n0);
}

// Too few tiles for all CUs: K split over workgroups, fp32 sums by position into part; the
// first split has the adapters too.
template <class C, bool KS, bool ORDERED, bool PIPE, int STAGES>
__global__ __launch_bounds__(C::THREADS, C::OCCUPANCY) void adapters_tile_split_kernel(AdapterParams p) {
    __shared__ __attribute__((aligned(1024))) char smem[AdapterTile<C, KS, ORDERED, STAGES>::LDS];
    const int tiles_n = (p.N + C::BN - 1) / C::BN, z = blockIdx.x % p.splits;
    const int m0 = (int)(blockIdx.x / p.splits / tiles_n) * C::BM, n0 = (int)(blockIdx.x / p.splits % tiles_n) * C::BN;
    if (m0 >= p.rows) return;
    int begin, end;
    split_range((p.K + C::BK - 1) / C::BK, p.splits, z, begin, end);
    const int k0 = begin * C::BK, K = (end * C::BK < p.K ? end * C::BK : p.K) - k0;
    AdapterTile<C, KS, ORDERED, STAGES> tile;
    tile.init(p, m0, p.rows - m0, k0, K > 0 ? K : 0, p.B + (KS ? k0 * p.ldb + n0 : n0 * p.ldb + k0) * C::ELEM, p.ldb,
              p.N - n0, smem);
    if constexpr (PIPE) tile.run_pipe();
    else tile.run_ring();
    const bool more = z == 0 && tile.adapters(p, m0, n0);
    float *part = p.part + ((int64_t)z * p.rows + m0) * p.N + n0;
    tile.store(reinterpret_cast<char *>(part), 0, p.N, p.rows - m0, p.N - n0, true, false);
    if (more) tile.left_out(p, m0, n0, [&](int m, int n, float sum) { part[(int64_t)m * p.N + n] += sum; });
}

// y from the splits' sums by position: a thread four neighbours of a row
template <int DT>
__global__ __launch_bounds__(256) void adapters_sum_kernel(AdapterParams p) {
    const int64_t quads = (p.N + 3) / 4, at = (int64_t)blockIdx.x * 256 + threadIdx.x, plane = (int64_t)p.rows * p.N;
    if (at >= quads * p.rows) return;
    const int pos = (int)(at / quads), c = (int)(at % quads) * 4, left = p.N - c;
    f32x4 y = {0, 0, 0, 0};
#pragma unroll 4
    for (int z = 0; z < p.splits; ++z)
        y += load4<DT_F32>(reinterpret_cast<const char *>(p.part), z * plane + (int64_t)pos * p.N + c, left, p.N % 4 == 0);
    store4<DT>(p.C, (int64_t)row_at(p, pos) * p.ldc + c, left, false, wide_rows<DT>(p.C, p.ldc), y);
}

// ---- the adapters' gradients ----------------------------------------------------------------
// C[g] = L[rows of g]^T . S[rows of g], L wide (M columns), S narrow (rank).  A workgroup
// takes kChunk positions of one adapter and a strip of L's columns a wave: stages of L as
// StreamB loads a matrix (32 rows by 128 columns, fp32 64), transposed in registers, the
// next one's loads in flight during the current one's products; S's rows of the chunk lie
// transposed in LDS, 16 JT of the rank.  An adapter of one chunk gets its result at once;
// else fp32 sums, rank x M of each chunk, go to the workspace: an adapter's first to place
// offsets[g] / kChunk (no other adapter of several chunks starts there), the further ones
// to their slots behind all of those.  Bound by the bytes of L while the rank is small; the
// sums are rank / 128 of its bytes in 16 bits, written and read again (8192 rows of 4096 and 4096
// bf16, two adapters: rank 16 55 us, 32 67, 64 92, 128 143), and above rank 32 a wave is alone on
// its SIMD.
constexpr int kChunk = 256;
constexpr int kWgradRank = 64;        // of the rank at a time

struct AdapterGradParams {
    // job 0: L = x, S = d_t -> d_A; job 1: L = d_y, S = t -> d_B
    const char *L[2], *S[2];
    char *C[2];
    int64_t ldl[2], lds[2], ldc[2], sC[2];
    int M[2];
    int wide_first[2];                 // C is M x rank (1) or rank x M (0)
    float *part[2];                    // [first chunks, then further ones][rank][M]
    const int32_t *offsets, *order;
    int adapters, rows, rank, c_f32;
    int strips[2], slots, rank_tiles;
};

// Four neighbours m .. m + 3 (left of them exist) of rank j of C[g].
template <int DT>
__device__ __forceinline__ void wgrad_store(const AdapterGradParams &p, int job, int g, int j, int m, int left, const f32x4 &x) {
    typedef typename ElemOf<DT>::type T;
    const int64_t at = (int64_t)g * p.sC[job], ld = p.ldc[job];
    const bool f32 = DT == DT_F32 || p.c_f32;
    if (!p.wide_first[job]) {
        const int64_t to = at + j * ld + m;
        const bool wide = ld % 4 == 0 && p.sC[job] % 4 == 0 && reinterpret_cast<uintptr_t>(p.C[job]) % (f32 ? 16 : 8) == 0;
        store4<DT>(p.C[job], to, left, p.c_f32, wide, x);
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if (e >= left) continue;
            const int64_t to = at + (m + e) * ld + j;
            if (f32) reinterpret_cast<float *>(p.C[job])[to] = x[e];
            else reinterpret_cast<T *>(p.C[job])[to] = (T)x[e];
        }
    }
}

template <int DT, int JT>
__global__ __launch_bounds__(256) void adapters_wgrad_kernel(AdapterGradParams p) {
    using Sh = StreamShape<DT, false>;
    typedef typename ElemOf<DT>::type T;
    typedef Chunk<DT> X;
    constexpr int E = Sh::E, PER = Sh::PER, PITCH = kChunk + PER, RANKS = 16 * JT;   // rows of S^T off the same banks
    __shared__ __attribute__((aligned(16))) T st[RANKS * PITCH];
    __shared__ int32_t row_of[kChunk];
    // workgroups: (job, strips of 4 x COLS columns, rank tile, slot)
    int id = blockIdx.x;
    const int per0 = p.strips[0] * p.rank_tiles * p.slots, job = id >= per0;
    if (job) id -= per0;
    const int strips = p.strips[job], strip = id % strips, rank_tile = id / strips % p.rank_tiles,
              block = id / strips / p.rank_tiles;
    int g;
    RowSpan span;
    if (!row_slot<kChunk>(p.offsets, p.adapters, p.rows, block - (p.adapters + 1), g, span) || g == p.adapters) return;
    const int rows = span.hi - span.lo, j0 = rank_tile * kWgradRank;
    const int ranks = p.rank - j0 < RANKS ? p.rank - j0 : RANKS;
    for (int k = threadIdx.x; k < kChunk; k += 256) {
        const int pos = span.lo + (k < rows ? k : 0);       // past the chunk its first again, times a zero of S
        row_of[k] = p.order ? row_in(p.order, pos, p.rows) : pos;
    }
    __syncthreads();
    for (int it = threadIdx.x; it < kChunk * (RANKS / PER); it += 256) {
        const int k = it % kChunk, j = it / kChunk * PER;
        X x;
        x.load(p.S[job], (int64_t)row_of[k] * p.lds[job] + j0 + j, k < rows ? ranks - j : 0);
#pragma unroll
        for (int e = 0; e < PER; ++e) st[(j + e) * PITCH + k] = x.x[e];
    }
    __syncthreads();
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, grp = lane / 16, c = lane % 16;
    const int m0 = (strip * 4 + wave) * Sh::COLS;
    if (m0 >= p.M[job]) return;
    f32x4 acc[JT][Sh::FRAGS];
#pragma unroll
    for (int j = 0; j < JT; ++j)
#pragma unroll
        for (int f = 0; f < Sh::FRAGS; ++f) acc[j][f] = f32x4{0, 0, 0, 0};
    const int left = p.M[job] - m0 - PER * c;
    const char *L = p.L[job] + (int64_t)(m0 + PER * c) * E;
    const int64_t ldl = p.ldl[job] * E;
    // Rows past the chunk meet zeros of S, so they may hold anything finite: its first row
    // does.  An infinity or NaN there would not stay in its own sums, so a last stage that
    // is cut loads zeros instead.
    auto fetch = [&](int k0, u32x4 (&q)[8], auto whole) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int k = k0 + (DT == DT_F32 ? 16 * (i / 4) + 4 * grp + i % 4 : 8 * grp + i);
            const char *at = L + row_of[k] * ldl;
            if constexpr (decltype(whole)::value) q[i] = *reinterpret_cast<const u32x4_unaligned *>(at);
            else q[i] = load_part<E, PART_ELEMENTS>(at, k < rows ? left : 0);
        }
    };
    auto multiply = [&](int k0, const u32x4 (&q)[8]) {
        if constexpr (DT == DT_F32) {
#pragma unroll
            for (int s = 0; s < 2; ++s)
#pragma unroll
                for (int j = 0; j < JT; ++j) {
                    const f32x4 x = *reinterpret_cast<const f32x4 *>(&st[(16 * j + c) * PITCH + k0 + 16 * s + 4 * grp]);
#pragma unroll
                    for (int e = 0; e < 4; ++e)
#pragma unroll
                        for (int f = 0; f < Sh::FRAGS; ++f) {
                            const uint32_t w = q[4 * s + e][f];
                            acc[j][f] = __builtin_amdgcn_mfma_f32_16x16x4f32(__builtin_bit_cast(float, w), x[e], acc[j][f],
                                                                            0, 0, 0);
                        }
                }
        } else {
            u32x4 f[8];
            transpose_square<2>(q, f);
#pragma unroll
            for (int j = 0; j < JT; ++j) {
                const u32x4 x = *reinterpret_cast<const u32x4 *>(&st[(16 * j + c) * PITCH + k0 + 8 * grp]);
#pragma unroll
                for (int i = 0; i < 8; ++i) mfma_chunk<DT>(f[i], x, acc[j][i]);
            }
        }
    };
    const int whole = p.M[job] - m0 >= Sh::COLS ? rows / Sh::K * Sh::K : 0;
    int k0 = 0;
    if (whole > 0) {
        u32x4 q0[8], q1[8];
        fetch(0, q0, std::true_type{});
        for (;;) {
            const bool more = k0 + Sh::K < whole;
            if (more) fetch(k0 + Sh::K, q1, std::true_type{});
            __builtin_amdgcn_sched_barrier(0);
            multiply(k0, q0);
            k0 += Sh::K;
            if (!more) break;
            for (int i = 0; i < 8; ++i) q0[i] = q1[i];
        }
    }
    for (; k0 < rows; k0 += Sh::K) {
        u32x4 q[8];
        fetch(k0, q, std::false_type{});
        multiply(k0, q);
    }
    // a lane holds, of rank j, the columns PER * (4 grp + v) + fragment: PER x 4 neighbours
    const int M = p.M[job], further = block - (p.adapters + 1);
    const RowSpan all = rows_of(p.offsets, g, p.adapters, p.rows);
    const bool alone = all.hi - all.lo <= kChunk, wide = M % 4 == 0;
    const int place = further < 0 ? all.lo / kChunk : (p.rows - 1) / kChunk + 1 + further;
    char *part = reinterpret_cast<char *>(p.part[job] + ((int64_t)place * p.rank + j0) * M);
#pragma unroll
    for (int j = 0; j < JT; ++j) {
        if (16 * j + c >= ranks) continue;
#pragma unroll
        for (int v = 0; v < 4; ++v)
#pragma unroll
            for (int f = 0; f < Sh::FRAGS; f += 4) {
                const int m = m0 + PER * (4 * grp + v) + f, n = M - m;
                const f32x4 x = {acc[j][f][v], acc[j][f + 1][v], acc[j][f + 2][v], acc[j][f + 3][v]};
                if (n <= 0) continue;
                if (alone) wgrad_store<DT>(p, job, g, j0 + 16 * j + c, m, n, x);
                else store4<DT_F32>(part, (int64_t)(16 * j + c) * M + m, n, true, wide, x);
            }
    }
}

// C[g] from the chunks' sums, in their order, for an adapter of several, and zeros for one
// without a row; a thread an element, threads along M (the sums' rows).
template <int DT>
__global__ __launch_bounds__(256) void adapters_wgrad_join_kernel(AdapterGradParams p) {
    typedef typename ElemOf<DT>::type T;
    const int job = blockIdx.z, g = blockIdx.y, M = p.M[job];
    const int64_t at = (int64_t)blockIdx.x * 256 + threadIdx.x, n = (int64_t)M * p.rank;
    if (at >= n) return;
    const int j = (int)(at / M), m = (int)(at % M);
    const RowSpan s = rows_of(p.offsets, g, p.adapters, p.rows);
    const int tiles = (s.hi - s.lo + kChunk - 1) / kChunk, first = s.lo / kChunk;
    if (tiles == 1) return;
    float sum = 0;
    if (tiles > 1) {
        const float *part = p.part[job] + at, *next = part + (int64_t)((p.rows - 1) / kChunk + 1 + first) * n;
        sum = part[first * n];
#pragma unroll 8
        for (int k = 0; k < tiles - 1; ++k) sum += next[k * n];
    }
    const int64_t to = (int64_t)g * p.sC[job] + (p.wide_first[job] ? m * p.ldc[job] + j : j * p.ldc[job] + m);
    if (DT == DT_F32 || p.c_f32) reinterpret_cast<float *>(p.C[job])[to] = sum;
    else reinterpret_cast<T *>(p.C[job])[to] = (T)sum;
}

}  // namespace tg
