// gated.hpp -- the gated pair of projections and the gradient of its gate, on block tiles
// and the LDS ring of grouped_ring.hpp, and the gate alone:
//
//   forward    u = A . Bg,  v = A . Bu,  h = act(u) * v        (U and V stored on request)
//   gradient   d_h = D . B,  d_u = d_h * v * act'(u),  d_v = d_h * act(u),  h = act(u) * v
//
// Forward: a workgroup's tile holds the same columns of both products, half of its MFMA
// column tiles each: the second operand is a pair, staged side by side, so that u and v
// of an element are in one wave and h costs no memory.  The tile of h is half as wide
// as the product's.  Gradient: the product's own tiles; u and v are read and the results
// written where d_h would have been.
//
// u, v, d_u and d_v are stored in the operands' type: they are operands of the products
// that follow (16 bits: one rounding of what the gate's gradient reads, one of what the
// products of the backward pass read; h is of the unrounded u and v).
//
// Measured, bf16, inputs that change from call to call: 8192 rows, 5632 x 2048 transposed,
// one expert, forward 323-335 us (1130-1170 TFLOP/s; a large library product 1319), bound by the
// matrix cores; 16384 rows of 8 uneven experts of 2048 x 2048 forward with u and v stored
// 270-285 us, of which about 30 are the stores; the gradient 200-206 us, of which the product
// alone is 125: u and v in, d_u and d_v out are 268 MB, 55 us at the rate of a large copy,
// and all CUs come to them at the same time.
#pragma once

#include <hip/hip_runtime.h>

#include "gate.hpp"
#include "grid.hpp"
#include "grouped_ring.hpp"

namespace tg {

struct GatedParams : GroupedParams {     // A, B (the gate's), C = H, ldc, N: columns of H
    const char *Bu;
    char *U, *V;                          // read by the gradient; U NULL: not stored
    char *dU, *dV;                        // C NULL: h not stored
    int64_t ldu, lddu;
    int act;
    // K split over workgroups (forward, few rows): fp32 sums of u and v, rows x N each,
    // split by split, in part
    float *part;
    int splits;
};

// The pair of second operands: MFMA tiles below T are the first's, the others the second's.
template <class V, bool KS, int T, int STAGES>
struct PairOperand {
    using O = RingOperand<V, KS, T>;
    static constexpr int PER = 2 * O::PER, REGION = 2 * O::REGION, PIECES = O::PIECES, REACH = O::REACH;
    O gate, up;
    __device__ __forceinline__ void init(const char *g, const char *u, int64_t ld, int left, int w, uint32_t lds, int lane,
                                         int wave) {
        gate.init(g, ld, left, w, lds, lane, wave);
        up.init(u, ld, left, w, lds + STAGES * O::REGION, lane, wave);
    }
    __device__ __forceinline__ void copy(int stage) {
        gate.copy(stage);
        up.copy(stage);
    }
    __device__ __forceinline__ void tail_load(int64_t k0, int K, u32x4 *tail) const {
        gate.tail_load(k0, K, tail);
        up.tail_load(k0, K, tail + O::PER);
    }
    __device__ __forceinline__ void tail_store(int stage, const u32x4 *tail) const {
        gate.tail_store(stage, tail);
        up.tail_store(stage, tail + O::PER);
    }
    __device__ __forceinline__ void read(int stage, int i, int q, u32x4 &f) const {
        if (i < T) gate.read(stage, i, q, f);
        else up.read(stage, i - T, q, f);
    }
};

template <class C> struct HalfCfg;
template <int DT, int BM, int BN, int WM, int WN, int MT>
struct HalfCfg<RingCfg<DT, BM, BN, WM, WN, MT>> {
    using type = RingCfg<DT, BM, BN / 2, WM, WN, MT>;
};
template <class C, bool KS, int STAGES>
using OperandPair = PairOperand<
    typename std::conditional<KS, typename HalfCfg<C>::type, typename SwapCfg<typename HalfCfg<C>::type>::type>::type, KS,
    C::TN / 2, STAGES>;

template <class C, bool B_KS, int STAGES>
struct GatedTile : GroupedTile<C, false, B_KS, STAGES, OperandA<C, false>, OperandPair<C, B_KS, STAGES>> {
    using Base = GroupedTile<C, false, B_KS, STAGES, OperandA<C, false>, OperandPair<C, B_KS, STAGES>>;
    static constexpr int HN = C::BN / 2, TH = C::TN / 2;

    __device__ __forceinline__ void init(const char *A, int64_t lda, int m_left, const char *Bg, const char *Bu,
                                         int64_t ldb, int n_left, int K, char *smem) {
        this->begin(K, !B_KS || n_left >= HN || n_left % C::CHUNK == 0);
        const uint32_t lds0 = lds_address(smem);
        this->b.init(Bg, Bu, ldb, n_left, (this->wave % C::WAVES_N) * (C::WTN / 2), lds0, this->lane, this->wave);
        this->a.init(A, lda, m_left, (this->wave / C::WAVES_N) * C::WTM, lds0 + STAGES * Base::OB::REGION, this->lane,
                     this->wave);
        this->acc.zero();
    }
    // u (FIRST 0) or v (TN / 2) in fp32
    template <int FIRST>
    __device__ __forceinline__ void store_sums(float *to, int64_t ld, int m_left, int n_left) const {
        const auto value = [&](auto i, auto j, auto v) {
            return this->acc.get(decltype(i)::value, FIRST + decltype(j)::value, decltype(v)::value);
        };
        TileStore<C, TH, decltype(value)>{value, this->lane, this->wave}.store(reinterpret_cast<char *>(to), 0, ld, m_left,
                                                                               n_left, true, false);
    }
};

// 16 bytes at any element boundary
typedef u32x4 __attribute__((aligned(2))) u32x4_unaligned;

// Elements of a row at p, of which `left` exist (16 bytes at most; fewer: the others 0).
template <int DT>
struct Chunk {
    typedef typename ElemOf<DT>::type T;
    static constexpr int PER = 16 / (int)sizeof(T);
    typedef T vec __attribute__((ext_vector_type(PER)));
    vec x;
    __device__ __forceinline__ void load(const char *p, int64_t at, int left) {
        const T *q = reinterpret_cast<const T *>(p) + at;
        x = vec{};
        if (left >= PER) {
            x = __builtin_bit_cast(vec, *reinterpret_cast<const u32x4_unaligned *>(q));
        } else {
#pragma unroll
            for (int e = 0; e < PER - 1; ++e)
                if (e < left) x[e] = q[e];
        }
    }
    // past: with the non-temporal hint (GroupedParams::past)
    __device__ __forceinline__ void store(char *p, int64_t at, int left, bool past) const {
        T *q = reinterpret_cast<T *>(p) + at;
        if (left >= PER) {
            u32x4_unaligned *to = reinterpret_cast<u32x4_unaligned *>(q);
            if (past) __builtin_nontemporal_store(__builtin_bit_cast(u32x4, x), to);
            else *to = __builtin_bit_cast(u32x4, x);
        } else {
#pragma unroll
            for (int e = 0; e < PER - 1; ++e)
                if (e < left) q[e] = x[e];
        }
    }
};

// A wave's accumulators as rows, through the LDS that the ring has left, in its own share
// of it, RI row tiles at a time: what follows the product is then a loop over 16-byte
// chunks of rows (straight-line code over the accumulators is 50 KB for the gradient, and
// waits for its instructions).  fp32; a row's 16-byte chunks are swapped by its number,
// which leaves the writes of a fragment without bank conflicts.
template <class C, class Tile>
struct WaveRows {
    static constexpr int CHUNKS = C::WTN / 4, SHARE = Tile::LDS / C::WAVES, ROW_TILE = 16 * C::WTN * 4;
    static constexpr int ri() {
        int r = C::TM;
        while (r * ROW_TILE > SHARE) r /= 2;
        return r;
    }
    static constexpr int RI = ri(), ROWS = 16 * RI, PASSES = C::TM / RI;
    static_assert(RI >= 1 && RI * PASSES == C::TM, "whole passes");
    uint32_t lds;
    int lane;
    __device__ __forceinline__ uint32_t place(int row, int chunk) const {
        return lds + (row * CHUNKS + (chunk ^ (row & (CHUNKS < 16 ? CHUNKS - 1 : 15)))) * 16;
    }
    template <int pass>
    __device__ __forceinline__ void put(const Tile &tile) const {
        static_for<0, C::TN, 1>([&](auto jc) {
            constexpr int j = decltype(jc)::value;
            // a row tile further is a constant, so one address a column tile, made here
            uint32_t at = place(lane % 16, 4 * j + lane / 16);
            asm volatile("" : "+v"(at));
            static_for<0, RI, 1>([&](auto ic) {
                constexpr int i = decltype(ic)::value, ai = pass * RI + i;
                const f32x4 v = {tile.acc.get(ai, j, 0), tile.acc.get(ai, j, 1), tile.acc.get(ai, j, 2),
                                 tile.acc.get(ai, j, 3)};
                *(__attribute__((address_space(3))) f32x4 *)(uintptr_t)(at + i * ROW_TILE) = v;
            });
        });
    }
    // N values of `row` from column `col` (a multiple of 4)
    template <int N>
    __device__ __forceinline__ void get(int row, int col, float (&f)[N]) const {
#pragma unroll
        for (int q = 0; q < N / 4; ++q) {
            const f32x4 v = *(const __attribute__((address_space(3))) f32x4 *)(uintptr_t)place(row, col / 4 + q);
#pragma unroll
            for (int e = 0; e < 4; ++e) f[4 * q + e] = v[e];
        }
    }
    // work(first row of the pass) for every pass, its rows in LDS
    template <class F>
    __device__ __forceinline__ void each(const Tile &tile, char *smem, const F &work) {
        lane = tile.lane;
        lds = lds_address(smem) + tile.wave * SHARE;
        block_barrier();                 // the ring's last readers are done
        static_for<0, PASSES, 1>([&](auto pc) {
            constexpr int pass = decltype(pc)::value;
            put<pass>(tile);
            wait_lds();
            work(pass * ROWS);
        });
    }
};

// split: of K, whose sums it stores instead (SPLIT; A, Bg, Bu and K are the split's)
template <class C, bool B_KS, bool PIPE, int STAGES, bool SPLIT = false>
__device__ __forceinline__ void run_gated(const GatedParams &p, char *smem, const RowTile &t, const char *A, const char *Bg,
                                          const char *Bu, int K, int64_t row, int split = 0) {
    GatedTile<C, B_KS, STAGES> tile;
    tile.init(A, p.lda, t.rows, Bg, Bu, p.ldb, p.N - t.n0, K, smem);
    if constexpr (PIPE) tile.run_pipe();
    else tile.run_ring();
    if constexpr (SPLIT) {
        if (p.splits > 1) {
            float *part = p.part + (2 * (int64_t)split * p.rows + row) * p.N + t.n0;
            tile.template store_sums<0>(part, p.N, t.rows, p.N - t.n0);
            tile.template store_sums<C::TN / 2>(part + (int64_t)p.rows * p.N, p.N, t.rows, p.N - t.n0);
            return;
        }
    }
    // a lane a chunk of h's columns: u in the first half of the wave's, v in the second
    typedef Chunk<C::DT> X;
    constexpr int PER = X::PER, HALF = C::WTN / 2, ITEMS = HALF / PER;
    WaveRows<C, GatedTile<C, B_KS, STAGES>> rows;
    const int m = (tile.wave / C::WAVES_N) * C::WTM, n = t.n0 + (tile.wave % C::WAVES_N) * HALF;
    constexpr int COUNT = rows.ROWS * ITEMS / 64;
    const bool whole = t.rows >= C::BM && p.N - t.n0 >= C::BN / 2;
    // a whole tile without a branch, four chunks at a time, their steps side by side
    auto pass = [&](int first, auto a, auto w) {
        constexpr bool WHOLE = decltype(w)::value;
        constexpr int BATCH = !WHOLE ? 1 : (COUNT < 4 ? COUNT : 4);
        static_assert(COUNT * 64 == rows.ROWS * ITEMS && COUNT % BATCH == 0, "whole batches");
#pragma unroll 1
        for (int batch = 0; batch < COUNT; batch += BATCH) {
            float u[BATCH][PER], v[BATCH][PER];
            X xu[BATCH], xv[BATCH], xh[BATCH];
#pragma unroll
            for (int k = 0; k < BATCH; ++k) {
                const int it = (batch + k) * 64 + tile.lane, r = it / ITEMS, c = it % ITEMS * PER;
                rows.get(r, c, u[k]);
                rows.get(r, HALF + c, v[k]);
            }
#pragma unroll
            for (int k = 0; k < BATCH; ++k)
#pragma unroll
                for (int e = 0; e < PER; ++e) {
                    xu[k].x[e] = (typename X::T)u[k][e];
                    xv[k].x[e] = (typename X::T)v[k][e];
                    xh[k].x[e] = (typename X::T)(gate_act<decltype(a)::value>(u[k][e]) * v[k][e]);
                }
#pragma unroll
            for (int k = 0; k < BATCH; ++k) {
                const int it = (batch + k) * 64 + tile.lane, r = it / ITEMS, c = it % ITEMS * PER;
                const int left = WHOLE ? PER : (m + first + r < t.rows ? p.N - n - c : 0);
                const int64_t to = row + m + first + r;
                if (p.U) {
                    xu[k].store(p.U, to * p.ldu + n + c, left, p.past);
                    xv[k].store(p.V, to * p.ldu + n + c, left, p.past);
                }
                xh[k].store(p.C, to * p.ldc + n + c, left, p.past);
            }
        }
    };
    rows.each(tile, smem, [&](int first) {
        with_act(p.act, [&](auto a) {
            if (whole) pass(first, a, std::true_type{});
            else pass(first, a, std::false_type{});
        });
    });
}

// P: the configuration of the pieces (C itself: none), as in grouped_tile_kernel.
template <class C, class P, bool B_KS, bool PIPE, int STAGES>
__global__ __launch_bounds__(C::THREADS, C::OCCUPANCY) void gated_tile_kernel(GatedParams p) {
    constexpr bool PIECES = !std::is_same<C, P>::value;
    __shared__ __attribute__((aligned(1024))) char smem[GatedTile<C, B_KS, STAGES>::LDS];
    RowTile t;
    if (!row_tile<C::BM, C::BN / 2, PIECES>(p, t)) return;
    const bool dead = t.g == p.experts;
    const int64_t row = t.lo + t.m0;
    const char *A = p.A + row * p.lda * C::ELEM;
    const int64_t b = ((dead ? 0 : (int64_t)t.g * p.sB) + (B_KS ? (int64_t)t.n0 : t.n0 * p.ldb)) * C::ELEM;
    const int K = dead ? 0 : p.K;
    if (PIECES && t.piece) run_gated<P, B_KS, PIPE, STAGES>(p, smem, t, A, p.B + b, p.Bu + b, K, row);
    else run_gated<C, B_KS, PIPE, STAGES>(p, smem, t, A, p.B + b, p.Bu + b, K, row);
}

// The stages (or K tiles) of split z of `splits`.
__device__ __forceinline__ void split_range(int stages, int splits, int z, int &begin, int &end) {
    begin = (int)((int64_t)stages * z / splits);
    end = (int)((int64_t)stages * (z + 1) / splits);
}

// Few rows an expert, but too many to take the weights straight to registers for: tiles of
// BM rows by row_slot, K split over workgroups.  grid: (column tiles x splits) x row tiles.
template <class C, bool B_KS, int STAGES>
__global__ __launch_bounds__(C::THREADS, C::OCCUPANCY) void gated_split_kernel(GatedParams p) {
    __shared__ __attribute__((aligned(1024))) char smem[GatedTile<C, B_KS, STAGES>::LDS];
    const int z = blockIdx.x % p.splits;
    RowTile t;
    RowSpan span;
    t.n0 = (int)(blockIdx.x / p.splits) * (C::BN / 2);
    if (!row_slot<C::BM>(p.offsets, p.experts, p.rows, slot_of(p.experts), t.g, span)) return;
    const bool dead = t.g == p.experts;
    const int64_t row = span.lo;
    t.rows = span.hi - span.lo;
    int begin = 0, end = 0;
    if (!dead) split_range((p.K + C::BK - 1) / C::BK, p.splits, z, begin, end);
    const int k0 = begin * C::BK, K = (end * C::BK < p.K ? end * C::BK : p.K) - k0;
    const char *A = p.A + (row * p.lda + k0) * C::ELEM;
    const int64_t b = ((dead ? 0 : (int64_t)t.g * p.sB) + (B_KS ? k0 * p.ldb + t.n0 : t.n0 * p.ldb + k0)) * C::ELEM;
    run_gated<C, B_KS, false, STAGES, true>(p, smem, t, A, p.B + b, p.Bu + b, K > 0 ? K : 0, row, z);
}

// Four neighbours of a row, n of which exist.
template <int DT>
__device__ __forceinline__ f32x4 load4(const char *p, int64_t at, int left, bool wide) {
    typedef typename ElemOf<DT>::type T;
    typedef T t4 __attribute__((ext_vector_type(4)));
    const T *q = reinterpret_cast<const T *>(p) + at;
    f32x4 v = {0, 0, 0, 0};
    if (wide && left >= 4) {
        const t4 x = *reinterpret_cast<const t4 *>(q);
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = (float)x[e];
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (e < left) v[e] = (float)q[e];
    }
    return v;
}

// whether rows of `ld` elements at p take four values in one aligned access
template <int DT>
__device__ __forceinline__ bool wide_rows(const char *p, int64_t ld) {
    return ld % 4 == 0 && reinterpret_cast<uintptr_t>(p) % (DT == DT_F32 ? 16 : 8) == 0;
}

// Rows of no expert: zeros, u and v not read.
struct GateGrad {
    bool dead, wide_in, wide_out, wide_h;
};
template <int DT>
__device__ __forceinline__ GateGrad gate_grad_of(const GatedParams &p, bool dead) {
    return {dead, wide_rows<DT>(p.U, p.ldu) && wide_rows<DT>(p.V, p.ldu),
            wide_rows<DT>(p.dU, p.lddu) && wide_rows<DT>(p.dV, p.lddu), wide_rows<DT>(p.C, p.ldc)};
}
// d_h = dh at row r, columns n .. n + 3 (left of them exist): the gradients of u and v, and h
template <int DT, int ACT>
__device__ __forceinline__ void gate_grad4(const GatedParams &p, const GateGrad &how, int64_t r, int64_t n, int left,
                                           const f32x4 &dh) {
    f32x4 u = {0, 0, 0, 0}, v = {0, 0, 0, 0};
    if (!how.dead) {
        u = load4<DT>(p.U, r * p.ldu + n, left, how.wide_in);
        v = load4<DT>(p.V, r * p.ldu + n, left, how.wide_in);
    }
    f32x4 du, dv, h;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        float f, d;
        gate_both<ACT>(u[e], f, d);
        du[e] = dh[e] * v[e] * d;
        dv[e] = dh[e] * f;
        h[e] = f * v[e];
    }
    store4<DT>(p.dU, r * p.lddu + n, left, false, how.wide_out, du);
    store4<DT>(p.dV, r * p.lddu + n, left, false, how.wide_out, dv);
    if (p.C) store4<DT>(p.C, r * p.ldc + n, left, false, how.wide_h, h);
}

template <class C, bool B_KS, bool PIPE, int STAGES>
__device__ __forceinline__ void run_gate_grad(const GatedParams &p, char *smem, const RowTile &t, const char *A,
                                              const char *B, int K, int64_t row, bool dead) {
    GroupedTile<C, false, B_KS, STAGES> tile;
    tile.init(A, p.lda, t.rows, B, p.ldb, p.N - t.n0, K, smem);
    typedef Chunk<C::DT> X;
    constexpr int PER = X::PER, ITEMS = C::WTN / PER;
    WaveRows<C, GroupedTile<C, false, B_KS, STAGES>> rows;
    constexpr int COUNT = rows.ROWS * ITEMS / 64, WIDE = COUNT < 4 ? COUNT : 4;
    static_assert(COUNT * 64 == rows.ROWS * ITEMS && COUNT % WIDE == 0, "whole batches");
    const int m = (tile.wave / C::WAVES_N) * C::WTM, n = t.n0 + (tile.wave % C::WAVES_N) * C::WTN;
    const bool whole = t.rows >= C::BM && p.N - t.n0 >= C::BN && !dead;
    // Chunk `it` of a pass, and u and v there.  In a whole tile, without a branch, four at a
    // time; those of the next four are in flight during the current ones' work, of the
    // first during the product's last K tiles.
    auto fetch = [&](int first, int it, X &u, X &v, bool all) {
        const int r = it / ITEMS, c = it % ITEMS * PER;
        const int left = all ? PER : (m + first + r < t.rows && !dead ? p.N - n - c : 0);
        const int64_t at = (row + m + first + r) * p.ldu + n + c;
        u.load(p.U, at, left);
        v.load(p.V, at, left);
    };
    X u[WIDE], v[WIDE];
    if (whole) {
#pragma unroll
        for (int k = 0; k < WIDE; ++k) fetch(0, k * 64 + (int)(threadIdx.x & 63), u[k], v[k], true);
    }
    if constexpr (PIPE) tile.run_pipe();
    else tile.run_ring();
    auto pass = [&](int first, auto a, auto w) {
        constexpr bool WHOLE = decltype(w)::value;
        constexpr int BATCH = WHOLE ? WIDE : 1, BATCHES = COUNT / BATCH;
#pragma unroll 1
        for (int batch = 0; batch < BATCHES; ++batch) {
            X u1[BATCH], v1[BATCH], du[BATCH], dv[BATCH], h[BATCH];
            if constexpr (WHOLE) {
                if (batch + 1 < BATCHES || first + rows.ROWS < C::WTM) {       // the next pass's rows follow
#pragma unroll
                    for (int k = 0; k < BATCH; ++k) fetch(first, ((batch + 1) * BATCH + k) * 64 + tile.lane, u1[k], v1[k], true);
                }
            } else {
                fetch(first, batch * 64 + tile.lane, u[0], v[0], false);
            }
#pragma unroll
            for (int k = 0; k < BATCH; ++k) {
                const int it = (batch * BATCH + k) * 64 + tile.lane, r = it / ITEMS, c = it % ITEMS * PER;
                float dh[PER];
                rows.get(r, c, dh);
#pragma unroll
                for (int e = 0; e < PER; ++e) {
                    float f, d;
                    gate_both<decltype(a)::value>((float)u[k].x[e], f, d);
                    const float ve = (float)v[k].x[e];
                    du[k].x[e] = (typename X::T)(dh[e] * ve * d);
                    dv[k].x[e] = (typename X::T)(dh[e] * f);
                    h[k].x[e] = (typename X::T)(f * ve);
                }
            }
#pragma unroll
            for (int k = 0; k < BATCH; ++k) {
                const int it = (batch * BATCH + k) * 64 + tile.lane, r = it / ITEMS, c = it % ITEMS * PER;
                const int left = WHOLE ? PER : (m + first + r < t.rows ? p.N - n - c : 0);
                const int64_t at = row + m + first + r;
                du[k].store(p.dU, at * p.lddu + n + c, left, p.past);
                dv[k].store(p.dV, at * p.lddu + n + c, left, p.past);
                if (p.C) h[k].store(p.C, at * p.ldc + n + c, left, p.past);
            }
            if constexpr (WHOLE) {
#pragma unroll
                for (int k = 0; k < BATCH; ++k) {
                    u[k] = u1[k];
                    v[k] = v1[k];
                }
            }
        }
    };
    rows.each(tile, smem, [&](int first) {
        with_act(p.act, [&](auto a) {
            if (whole) pass(first, a, std::true_type{});
            else pass(first, a, std::false_type{});
        });
    });
}

template <class C, class P, bool B_KS, bool PIPE, int STAGES>
__global__ __launch_bounds__(C::THREADS, C::OCCUPANCY) void gate_grad_tile_kernel(GatedParams p) {
    constexpr bool PIECES = !std::is_same<C, P>::value;
    __shared__ __attribute__((aligned(1024))) char smem[GroupedTile<C, false, B_KS, STAGES>::LDS];
    RowTile t;
    if (!row_tile<C::BM, C::BN, PIECES>(p, t)) return;
    const bool dead = t.g == p.experts;
    const int64_t row = t.lo + t.m0;
    const char *A = p.A + row * p.lda * C::ELEM;
    const char *B = p.B + ((dead ? 0 : (int64_t)t.g * p.sB) + (B_KS ? (int64_t)t.n0 : t.n0 * p.ldb)) * C::ELEM;
    const int K = dead ? 0 : p.K;
    if (PIECES && t.piece) run_gate_grad<P, B_KS, PIPE, STAGES>(p, smem, t, A, B, K, row, dead);
    else run_gate_grad<C, B_KS, PIPE, STAGES>(p, smem, t, A, B, K, row, dead);
}

// The gate alone, on rows that another product gave (an adapted or a 4-bit one): h from u
// and v; d_u, d_v and h from d_h (A), u and v.  A thread 16 bytes of a row; bound by memory
// (8192 x 5632 bf16 50 us,
// 5.5 TB/s; the gradient 86 us, 5.4, with h 102).
template <int DT, bool GRAD>
__global__ __launch_bounds__(256) void gate_kernel(GatedParams p) {
    typedef Chunk<DT> X;
    const int64_t chunks = (p.N + X::PER - 1) / X::PER, at = (int64_t)wide_block() * 256 + threadIdx.x, r = at / chunks;
    if (r >= p.rows) return;
    const int64_t c = at % chunks * X::PER;
    const int left = p.N - (int)c;
    X u, v, dh, h, du, dv;
    u.load(p.U, r * p.ldu + c, left);
    v.load(p.V, r * p.ldu + c, left);
    if constexpr (GRAD) dh.load(p.A, r * p.lda + c, left);
    with_act(p.act, [&](auto a) {
#pragma unroll
        for (int e = 0; e < X::PER; ++e) {
            const float ue = (float)u.x[e], ve = (float)v.x[e];
            if constexpr (GRAD) {
                float f, d;
                gate_both<decltype(a)::value>(ue, f, d);
                du.x[e] = (typename X::T)((float)dh.x[e] * ve * d);
                dv.x[e] = (typename X::T)((float)dh.x[e] * f);
                h.x[e] = (typename X::T)(f * ve);
            } else {
                h.x[e] = (typename X::T)(gate_act<decltype(a)::value>(ue) * ve);
            }
        }
    });
    if constexpr (GRAD) {
        du.store(p.dU, r * p.lddu + c, left, p.past);
        dv.store(p.dV, r * p.lddu + c, left, p.past);
    }
    if (!GRAD || p.C) h.store(p.C, r * p.ldc + c, left, p.past);
}

}  // namespace tg
