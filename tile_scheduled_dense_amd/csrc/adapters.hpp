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
//  * Few rows (the bytes of W): one launch sums x . W (its columns in strips, K split over
//    workgroups) and x . A[g] (16 positions of one adapter a workgroup, K split) into fp32
//    partial sums, a second one adds them and t . B[g].
//  * Many rows: t first (16 positions a workgroup, rounded once to the inputs' type: it
//    is the second product's operand), then the block tiles of grouped_ring.hpp over
//    positions, whose contraction goes on through t and the B[g] of every adapter that
//    has positions in the tile, the others' rows of t being zeros.
//  * Gradients: 16-bit and fp32 products whose contraction is an adapter's rows, the wide
//    operand straight from memory to registers, the narrow one transposed in LDS; a
//    workgroup takes a chunk of an adapter's rows, a second launch adds the chunks in
//    their order.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "few_rows.hpp"

namespace tg {

struct AdapterParams : GroupedParams {   // A: x, B: W, C: y; experts: adapters; sB unused
    const char *down, *up;                // the adapters' A and B
    const float *scales;                  // NULL: 1
    const int32_t *order;
    char *T;                              // NULL: not stored
    char *low;                            // many rows: t of dtype by position, rows of ld_low
    float *part, *part_t;                 // few rows: sums of x . W (by row), of x . A[g] (by position)
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
    few_range(stages, p.t_splits, split, begin, end);
    few_sum<DT, TRANS>(of, row, p.K, p.K % S::PER == 0 && (TRANS || p.rank % S::PER == 0), begin + wave, waves, end, lane,
                       acc);
#pragma unroll
    for (int j = 0; j < S::FRAGS; ++j) lds[(wave * S::FRAGS + j) * 64 + lane] = acc[j];
    __syncthreads();
    return true;
}

// ---- few rows -------------------------------------------------------------------------------
// Workgroups below `base`: x . W (strips x splits x tiles of 16 rows); behind them x . A[g].
template <int DT, bool TRANS>
__global__ __launch_bounds__(512) void adapters_few_kernel(AdapterParams p, int base, int row_tiles, int strips_t) {
    using S = StreamShape<DT, TRANS>;
    extern __shared__ f32x4 stream_lds[];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int lane = threadIdx.x & 63, waves = blockDim.x >> 6;
    int id = blockIdx.x;
    if (id >= base) {
        id -= base;
        const int split = id % p.t_splits, strip = id / p.t_splits % strips_t, slot = id / p.t_splits / strips_t;
        int g;
        RowSpan span;
        if (!shrink_sum<DT, TRANS>(p, strip, slot - (p.experts + 1), split, stream_lds, g, span) || g == p.experts) return;
        const int n0 = strip * S::COLS;
        for (int it = threadIdx.x; it < S::FRAGS * 64; it += blockDim.x) {
            int m, n;
            const f32x4 v = few_item<DT, TRANS>(stream_lds, waves, it, m, n);
            const int left = p.rank - n0 - n;
            if (m < span.hi - span.lo && left > 0)
                store4<DT_F32>(reinterpret_cast<char *>(p.part_t),
                               ((int64_t)split * p.rows + span.lo + m) * p.rank + n0 + n, left, true, p.rank % 4 == 0, v);
        }
        return;
    }
    const int z = id % p.splits, tile = id / p.splits % row_tiles, n0 = id / p.splits / row_tiles * S::COLS;
    const int r0 = 16 * tile, stages = (p.K + S::K - 1) / S::K;
    const OneStrip<DT, TRANS> of = {p.B + (TRANS ? n0 * p.ldb : (int64_t)n0) * S::E, p.ldb, p.N - n0};
    const char *row = r0 + lane % 16 < p.rows ? p.A + (int64_t)(r0 + lane % 16) * p.lda * S::E : nullptr;
    f32x4 acc[S::FRAGS];
#pragma unroll
    for (int j = 0; j < S::FRAGS; ++j) acc[j] = f32x4{0, 0, 0, 0};
    int begin, end;
    few_range(stages, p.splits, z, begin, end);
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

// y and t of a position from the sums (workgroups: position by position): a thread four neighbours of y.  t in LDS,
// in fp32, 256 of the rank at a time.
constexpr int kJoinRank = 256;
template <int DT, bool TRANS>
__global__ __launch_bounds__(256) void adapters_join_kernel(AdapterParams p) {
    typedef typename ElemOf<DT>::type E;
    __shared__ float t[kJoinRank];
    const int parts = (p.N + 1023) / 1024, pos = blockIdx.x / parts, part = blockIdx.x % parts;
    const int g = group_of(p.offsets, p.experts, pos);
    const int64_t r = row_at(p, pos);
    const int c = 4 * (part * 256 + (int)threadIdx.x), left = p.N - c;
    f32x4 y = {0, 0, 0, 0};
    if (left > 0)
        for (int z = 0; z < p.splits; ++z)
            y += load4<DT_F32>(reinterpret_cast<const char *>(p.part), ((int64_t)z * p.rows + r) * p.N + c, left, p.N % 4 == 0);
    const bool has = g < p.experts;
    const float scale = has ? (p.scales ? p.scales[g] : 1.0f) : 0.0f;
    const E *up = reinterpret_cast<const E *>(p.up) + (has ? (int64_t)g * p.s_up : 0);
    for (int k0 = 0; k0 < p.rank; k0 += kJoinRank) {
        const int n = p.rank - k0 < kJoinRank ? p.rank - k0 : kJoinRank;
        __syncthreads();
        for (int k = threadIdx.x; k < n; k += 256) {
            float s = 0;
            if (has)
                for (int z = 0; z < p.t_splits; ++z) s += p.part_t[((int64_t)z * p.rows + pos) * p.rank + k0 + k];
            s *= scale;
            if (!has) s = 0;
            t[k] = s;
            if (p.T && part == 0) reinterpret_cast<E *>(p.T)[r * p.ldt + k0 + k] = (E)s;
        }
        __syncthreads();
        if (!has || left <= 0) continue;
        for (int k = 0; k < n; ++k) {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (e < left)
                    y[e] = __builtin_fmaf(t[k], (float)(TRANS ? up[(int64_t)(c + e) * p.ld_up + k0 + k]
                                                              : up[(int64_t)(k0 + k) * p.ld_up + c + e]), y[e]);
        }
    }
    if (left > 0) store4<DT>(p.C, r * p.ldc + c, left, false, wide_rows<DT>(p.C, p.ldc), y);
}

// ---- many rows ------------------------------------------------------------------------------
// t by position, of dtype, into low (its rows' rest up to ld_low zeros), and into T.
template <int DT, bool TRANS>
__global__ __launch_bounds__(512) void shrink_kernel(AdapterParams p) {
    using S = StreamShape<DT, TRANS>;
    extern __shared__ f32x4 stream_lds[];
    const int waves = blockDim.x >> 6, n0 = blockIdx.x * S::COLS;
    int g;
    RowSpan span;
    if (!shrink_sum<DT, TRANS>(p, blockIdx.x, slot_of(p.experts), 0, stream_lds, g, span)) return;
    const bool has = g < p.experts;
    const float scale = has && p.scales ? p.scales[g] : 1.0f;
    for (int it = threadIdx.x; it < S::FRAGS * 64; it += blockDim.x) {
        int m, n;
        f32x4 v = few_item<DT, TRANS>(stream_lds, waves, it, m, n);
        const int left = p.rank - n0 - n;
        if (m >= span.hi - span.lo) continue;
        v *= scale;
        if (!has) v = f32x4{0, 0, 0, 0};
        const int pos = span.lo + m, low_left = (int)p.ld_low - n0 - n;
        if (low_left > 0) store4<DT>(p.low, (int64_t)pos * p.ld_low + n0 + n, low_left, false, true, v);
        if (p.T && left > 0) store4<DT>(p.T, (int64_t)row_at(p, pos) * p.ldt + n0 + n, left, false, wide_rows<DT>(p.T, p.ldt), v);
    }
}

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

template <class C, bool KS, bool ORDERED, int STAGES>
struct AdapterTile
    : GroupedTile<C, false, KS, STAGES,
                  typename std::conditional<ORDERED, OrderedOperand<C, C::TM>, OperandA<C, false>>::type, OperandB<C, KS>> {
    using OA = typename std::conditional<ORDERED, OrderedOperand<C, C::TM>, OperandA<C, false>>::type;
    using OB = OperandB<C, KS>;

    __device__ __forceinline__ void init(const AdapterParams &p, int m0, int n0, char *smem) {
        const int m_left = p.rows - m0, n_left = p.N - n0;
        this->begin(p.K, !KS || n_left >= C::BN || n_left % C::CHUNK == 0);
        const uint32_t lds0 = lds_address(smem);
        this->b.init(p.B + (KS ? (int64_t)n0 : n0 * p.ldb) * C::ELEM, p.ldb, n_left, (this->wave % C::WAVES_N) * C::WTN, lds0,
                     this->lane, this->wave);
        const int w = (this->wave / C::WAVES_N) * C::WTM;
        if constexpr (ORDERED)
            this->a.init(p.A, p.lda, m_left, w, lds0 + STAGES * OB::REGION, this->lane, this->wave, p.order + m0, p.rows);
        else
            this->a.init(p.A + (int64_t)m0 * p.lda * C::ELEM, p.lda, m_left, w, lds0 + STAGES * OB::REGION, this->lane,
                         this->wave);
        this->acc.zero();
    }

    // The contraction goes on: t . B[g] for every adapter with positions in the tile, in
    // K tiles of the rank through registers, one at a time (an adapter of 32 and less is
    // one), other adapters' rows and what lies past the rank as zeros.
    __device__ __forceinline__ void adapters(const AdapterParams &p, int m0, int n0) {
        if (this->nk == 0) return;                 // t is zero too
        const int m_end = m0 + C::BM < p.rows ? m0 + C::BM : p.rows;
        const int last = __builtin_amdgcn_readfirstlane(group_of(p.offsets, p.experts, m_end - 1));
        for (int g = __builtin_amdgcn_readfirstlane(group_of(p.offsets, p.experts, m0)); g <= last && g < p.experts; ++g) {
            const RowSpan s = rows_of(p.offsets, g, p.experts, p.rows);
            const int lo = __builtin_amdgcn_readfirstlane(s.lo) - m0, hi = __builtin_amdgcn_readfirstlane(s.hi) - m0;
            if (hi <= 0 || lo >= C::BM || hi <= lo) continue;
            const rsrc_t rt = make_rsrc(p.low + (int64_t)m0 * p.ld_low * C::ELEM);
            const char *up = p.up + ((int64_t)g * p.s_up + (KS ? (int64_t)n0 : n0 * p.ld_up)) * C::ELEM;
            for (int k0 = 0; k0 < p.rank; k0 += C::BK) {
                u32x4 ta[OA::PER], tb[OB::PER];
#pragma unroll
                for (int d = 0; d < OA::PER; ++d) {
                    const int x = this->a.x[d], k = k0 + this->a.k[d];
                    const bool in = x >= lo && x < hi && x < m_end - m0 && k < p.ld_low;
                    ta[d] = bload16(rt, in ? (x * (int)p.ld_low + k) * C::ELEM : kOutOfRange, 0);
                }
                const rsrc_t rb = make_rsrc(up + (int64_t)k0 * (KS ? p.ld_up : 1) * C::ELEM);
#pragma unroll
                for (int d = 0; d < OB::PER; ++d) {
                    const int k_left = p.rank - k0 - this->b.k[d], x_left = this->b.left - this->b.x[d];
                    const int run = KS ? x_left : k_left, other = KS ? k_left : x_left;
                    const int n = other <= 0 || run <= 0 ? 0 : (run < C::CHUNK ? run : C::CHUNK);
                    const int at = KS ? this->b.k[d] * (int)p.ld_up + this->b.x[d] : this->b.x[d] * (int)p.ld_up + this->b.k[d];
                    tb[d] = bload16_n<C::ELEM>(rb, n > 0 ? at * C::ELEM : 0, 0, n);
                }
                block_barrier();                   // the copy's last readers are done
                this->a.tail_store(0, ta);
                this->b.tail_store(0, tb);
                wait_lds();
                block_barrier();
                u32x4 fa[C::TM], fb[C::TN];
#pragma unroll
                for (int r = 0; r < AdapterTile::READS; ++r) this->read_piece(0, r, fa, fb);
                static_for<0, AdapterTile::NMFMA, 1>(
                    [&](auto q) { this->template mma<false, decltype(q)::value>(fa, fb); });
                wait_lds();
            }
        }
        this->acc.settle();
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

template <class C, bool KS, bool ORDERED, bool PIPE, int STAGES>
__device__ __forceinline__ void run_adapters(const AdapterParams &p, char *smem, int m0, int n0) {
    AdapterTile<C, KS, ORDERED, STAGES> tile;
    tile.init(p, m0, n0, smem);
    if constexpr (PIPE) tile.run_pipe();
    else tile.run_ring();
    tile.adapters(p, m0, n0);
    tile.store_rows(p, m0, n0);
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

// ---- the adapters' gradients ----------------------------------------------------------------
// C[g] = L[rows of g]^T . S[rows of g], L wide (M columns), S narrow (rank).  A workgroup
// takes kChunk positions of one adapter and, a wave each, strips of L's columns: stages
// of L as StreamB loads a matrix (32 or 16... rows of k by 128 or 64 columns), transposed
// in registers; S's rows of the chunk lie transposed in LDS.  fp32 sums, rank x M of each
// chunk, go to the workspace.
constexpr int kChunk = 256;
constexpr int kWgradRank = 64;        // of the rank at a time

struct AdapterGradParams {
    // job 0: L = x, S = d_t -> d_A; job 1: L = d_y, S = t -> d_B
    const char *L[2], *S[2];
    char *C[2];
    int64_t ldl[2], lds[2], ldc[2], sC[2];
    int M[2];
    int wide_first[2];                 // C is M x rank (1) or rank x M (0)
    float *part[2];                    // [workgroup of kChunk][rank][M]
    const int32_t *offsets, *order;
    int adapters, rows, rank, c_f32;
    int strips[2], slots, rank_tiles;
};

template <int DT>
__global__ __launch_bounds__(256) void adapters_wgrad_kernel(AdapterGradParams p) {
    using Sh = StreamShape<DT, false>;
    typedef typename ElemOf<DT>::type T;
    constexpr int E = Sh::E, PER = Sh::PER, PITCH = kChunk + 16 / E;      // rows of S^T off the same banks
    constexpr int JT = kWgradRank / 16;
    __shared__ __attribute__((aligned(16))) T st[kWgradRank * PITCH];
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
    const int ranks = p.rank - j0 < kWgradRank ? p.rank - j0 : kWgradRank;
    for (int k = threadIdx.x; k < kChunk; k += 256)
        row_of[k] = k < rows ? (p.order ? row_in(p.order, span.lo + k, p.rows) : span.lo + k) : 0;
    __syncthreads();
    const T *S = reinterpret_cast<const T *>(p.S[job]);
    for (int it = threadIdx.x; it < kChunk * kWgradRank; it += 256) {
        const int j = it % kWgradRank, k = it / kWgradRank;
        st[j * PITCH + k] = j < ranks && k < rows ? S[row_of[k] * p.lds[job] + j0 + j] : (T)0.0f;
    }
    __syncthreads();
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, grp = lane / 16, c = lane % 16;
    const int m0 = (strip * 4 + wave) * Sh::COLS, left = p.M[job] - m0 - PER * c;
    if (m0 >= p.M[job]) return;
    f32x4 acc[JT][Sh::FRAGS];
#pragma unroll
    for (int j = 0; j < JT; ++j)
#pragma unroll
        for (int f = 0; f < Sh::FRAGS; ++f) acc[j][f] = f32x4{0, 0, 0, 0};
    const char *L = p.L[job] + (int64_t)(m0 + PER * c) * E;
    const int64_t ldl = p.ldl[job] * E;
    for (int k0 = 0; k0 < rows; k0 += Sh::K) {
        u32x4 q[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int k = k0 + (DT == DT_F32 ? 16 * (i / 4) + 4 * grp + i % 4 : 8 * grp + i);
            q[i] = load_part<E, PART_ELEMENTS>(L + row_of[k < rows ? k : 0] * ldl, k < rows ? left : 0);
        }
        if constexpr (DT == DT_F32) {
#pragma unroll
            for (int s = 0; s < 2; ++s)
#pragma unroll
                for (int j = 0; j < JT; ++j) {
                    if (16 * j >= ranks) continue;
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
                if (16 * j >= ranks) continue;
                const u32x4 x = *reinterpret_cast<const u32x4 *>(&st[(16 * j + c) * PITCH + k0 + 8 * grp]);
#pragma unroll
                for (int i = 0; i < 8; ++i) mfma_chunk<DT>(f[i], x, acc[j][i]);
            }
        }
    }
    // a lane holds, of rank j, the columns PER * (4 grp + v) + fragment: PER x 4 neighbours
    float *part = p.part[job] + ((int64_t)block * p.rank + j0) * p.M[job];
    const bool wide = p.M[job] % 4 == 0;
#pragma unroll
    for (int j = 0; j < JT; ++j) {
        if (16 * j + c >= ranks) continue;
#pragma unroll
        for (int v = 0; v < 4; ++v)
#pragma unroll
            for (int f = 0; f < Sh::FRAGS; f += 4) {
                const int m = m0 + PER * (4 * grp + v) + f, n = p.M[job] - m;
                const f32x4 x = {acc[j][f][v], acc[j][f + 1][v], acc[j][f + 2][v], acc[j][f + 3][v]};
                if (n > 0)
                    store4<DT_F32>(reinterpret_cast<char *>(part), (int64_t)(16 * j + c) * p.M[job] + m, n, true, wide, x);
            }
    }
}

// C[g] from the chunks' sums, in their order; a thread an element, zeros for an adapter
// without a row.
template <int DT>
__global__ __launch_bounds__(256) void adapters_wgrad_join_kernel(AdapterGradParams p) {
    typedef typename ElemOf<DT>::type T;
    const int job = blockIdx.z, g = blockIdx.y, M = p.M[job];
    const int64_t at = (int64_t)blockIdx.x * 256 + threadIdx.x, n = (int64_t)M * p.rank;
    if (at >= n) return;
    // consecutive threads along C's rows
    const int j = p.wide_first[job] ? (int)(at % p.rank) : (int)(at / M), m = p.wide_first[job] ? (int)(at / p.rank) : (int)(at % M);
    const RowSpan s = rows_of(p.offsets, g, p.adapters, p.rows);
    const float *part = p.part[job] + (int64_t)j * M + m;
    float sum = 0;
    for (int k = 0; s.lo + k * kChunk < s.hi; ++k) {
        const int block = k == 0 ? g : p.adapters + 1 + s.lo / kChunk + k - 1;
        sum += part[(int64_t)block * n];
    }
    const int64_t to = (int64_t)g * p.sC[job] + (p.wide_first[job] ? m * p.ldc[job] + j : j * p.ldc[job] + m);
    if (DT == DT_F32 || p.c_f32) reinterpret_cast<float *>(p.C[job])[to] = sum;
    else reinterpret_cast<T *>(p.C[job])[to] = (T)sum;
}

}  // namespace tg
