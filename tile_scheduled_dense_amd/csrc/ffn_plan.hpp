// ffn_plan.hpp -- which kernels an operator of a feed-forward block takes, their grids and
// their workspace: host arithmetic on sizes and types alone, shared by the launches
// (gated_kernels.hpp, adapters_kernels.hpp) and the C ABI (ffn.hip).
#pragma once

#include <hip/hip_runtime.h>

#include "adapters.hpp"
#include "experts_plan.hpp"

namespace tg {

// Waves of a workgroup that splits K (plan_stream).
inline int few_waves(int64_t stages) { return stages >= 16 ? 8 : (stages >= 8 ? 4 : 2); }

// Splits of K over workgroups, of which `groups` are at work without: until there are
// `enough`, at least `least` stages each.
inline int few_splits(int64_t groups, int64_t enough, int64_t stages, int64_t least) {
    int s = 1;
    while (groups * s * 2 <= enough && stages >= least * s * 2) s *= 2;
    return s;
}

// ---- the gated pair -----------------------------------------------------------------------
struct GatedPlan {
    int splits;                  // of K over workgroups; 0: block tiles, which are not split
    ProductPlan product;
};

template <int DT, bool TRANS>
GatedPlan plan_gated_as(int64_t experts, int64_t rows, int64_t N, int64_t K) {
    using S = StreamShape<DT, TRANS>;
    GatedPlan p = {};
    const int64_t used = rows < experts ? rows : experts, mean = cdiv(rows, experts), each = cdiv(rows, used);
    if (N < kNarrow || (mean <= 16 && (TRANS || DT == DT_F32))) {
        const int64_t cols = TwoStrips<DT, TRANS>::COLS, stages = cdiv(K, S::K);
        const int waves = few_waves(stages);
        p.splits = few_splits(cdiv(N, cols) * used * cdiv(each, 16), 256, stages, waves);
        p.product = plan_of(TG_EXPERTS_STREAM, 16, (int)cols, waves, cdiv(N, cols) * p.splits,
                            tiles_and_slots(rows, experts, 16));
        return p;
    }
    const int64_t strips = cdiv(N, 64) * used;
    const bool split = mean <= 64 || (DT != DT_F32 && mean <= 128 && strips <= 128);
    if (split || (DT != DT_F32 && cdiv(rows, 128) * cdiv(N, 64) <= 400)) {
        p.splits = split ? few_splits(strips, 256, cdiv(K, 64 / S::E), 8) : 1;
        p.product = plan_of(TG_EXPERTS_TILES, 64, 64, 4, cdiv(N, 64) * p.splits, tiles_and_slots(rows, experts, 64));
        return p;
    }
    const int64_t tiles = cdiv(rows, 256) * cdiv(N, 128);
    if (DT == DT_F32) p.product = plan_tiles(experts, rows, N, 64, 64, false, true, 4);
    else if (K >= kLong && tiles >= 128) p.product = plan_tiles(experts, rows, N, 256, 128, true, true, 4);
    else p.product = plan_tiles(experts, rows, N, 128, 64, false, false, 3);
    return p;
}
template <int DT>
GatedPlan plan_gated(bool transposed, int64_t experts, int64_t rows, int64_t N, int64_t K) {
    return transposed ? plan_gated_as<DT, true>(experts, rows, N, K) : plan_gated_as<DT, false>(experts, rows, N, K);
}
inline int64_t gated_workspace(const GatedPlan &p, int64_t rows, int64_t N) {
    return p.splits > 1 ? p.splits * 2 * rows * N * 4 : 0;
}

// The gate's gradient: the products' own rule (plan_grouped_as), but the smaller tiles of 16
// bits are smaller still.
template <int DT, bool TRANS>
ProductPlan plan_gate_grad_as(int64_t experts, int64_t rows, int64_t N, int64_t K) {
    const ProductPlan p = plan_grouped_as<DT, TRANS>(experts, rows, N, K);
    if (DT == DT_F32 || p.info.kernel != TG_EXPERTS_TILES || p.info.tile_m == 256) return p;
    return plan_tiles(experts, rows, N, 64, cdiv(rows, 64) * cdiv(N, 128) <= 512 ? 64 : 128, false, false, 4);
}

template <int DT>
ProductPlan plan_gate_grad(bool transposed, int64_t experts, int64_t rows, int64_t N, int64_t K) {
    return transposed ? plan_gate_grad_as<DT, true>(experts, rows, N, K) : plan_gate_grad_as<DT, false>(experts, rows, N, K);
}

// ---- adapters -------------------------------------------------------------------------------
// Up to so many rows a projection's columns and its adapters' share one launch, and another
// adds them up.
constexpr int64_t kAdapterFew = 64;

enum { ADAPTERS_STREAM = 0, ADAPTERS_SPLIT = 1, ADAPTERS_TILES = 2 };
struct AdapterPlan {
    int form;
    int splits, t_splits;        // of K: x . W, x . A[g]
    int64_t ld_low;              // tiles: t's row length
    int64_t part_bytes, part_t_bytes, bytes;   // workspace: sums of x . W, of x . A[g], all
    ProductPlan product;         // ADAPTERS_STREAM, _SPLIT: without the workgroups of x . A[g]
    ProductPlan low;             // x . A[g]
};

template <int DT, bool TRANS>
AdapterPlan plan_adapters_as(int64_t adapters, int64_t rows, int64_t N, int64_t K, int64_t rank) {
    using S = StreamShape<DT, TRANS>;
    AdapterPlan p = {};
    const int64_t stages = cdiv(K, S::K), k_tiles = cdiv(K, 64 / S::E);
    p.splits = p.t_splits = 1;
    if (rows <= kAdapterFew || N < kNarrow) {
        const bool stream = N < kNarrow || (rows <= 16 && (TRANS || DT == DT_F32));
        const int waves = 4;
        p.form = stream ? ADAPTERS_STREAM : ADAPTERS_SPLIT;
        const int64_t strips = cdiv(N, stream ? S::COLS : 64), tiles = strips * cdiv(rows, stream ? 16 : 64);
        p.splits = stream ? few_splits(tiles, 512, stages, waves) : few_splits(tiles, 256, k_tiles, 8);
        p.t_splits = few_splits(cdiv(rank, S::COLS), 8, stages, waves);
        p.part_bytes = round_up(p.splits * rows * N * 4, 16);
        p.part_t_bytes = round_up(p.t_splits * rows * rank * 4, 16);
        p.product = plan_of(stream ? TG_EXPERTS_STREAM : TG_EXPERTS_TILES, stream ? 16 : 64, stream ? S::COLS : 64, waves,
                            tiles * p.splits);
        p.low = plan_of(TG_EXPERTS_STREAM, 16, S::COLS, waves,
                        cdiv(rank, S::COLS) * p.t_splits * tiles_and_slots(rows, adapters, 16));
    } else {
        p.form = ADAPTERS_TILES;
        p.ld_low = round_up(rank, S::PER);
        p.t_splits = few_splits(cdiv(rows, 64) * cdiv(rank, 64), 512, k_tiles, 8);
        p.part_t_bytes = round_up(p.t_splits * rows * rank * 4, 16);
        p.low = plan_of(TG_EXPERTS_TILES, 64, 64, 4, cdiv(rank, 64) * p.t_splits, tiles_and_slots(rows, adapters, 64));
        const int64_t tiles = cdiv(rows, 256) * cdiv(N, 256);
        if (DT == DT_F32) p.product = plan_tiles(1, rows, N, 64, 64, false, true, 4);
        else if (K >= kLong && tiles >= 128) p.product = plan_tiles(1, rows, N, 256, 256, true, true, 4);
        else p.product = plan_tiles(1, rows, N, 128, 128, false, false, 3);
        if (p.product.info.tile_m < 256) {
            p.splits = few_splits(p.product.gx, 512, k_tiles, 16);
            if (p.splits > 1) p.part_bytes = round_up(p.splits * rows * N * 4, 16);
            const bool pipeline = p.product.info.pipeline;
            p.product = plan_of(TG_EXPERTS_TILES, p.product.info.tile_m, p.product.info.tile_n, 4, p.product.gx * p.splits);
            p.product.info.pipeline = pipeline;
        }
    }
    p.bytes = p.part_bytes + p.part_t_bytes + rows * p.ld_low * S::E;
    return p;
}
template <int DT>
AdapterPlan plan_adapters(bool transposed, int64_t adapters, int64_t rows, int64_t N, int64_t K, int64_t rank) {
    return transposed ? plan_adapters_as<DT, true>(adapters, rows, N, K, rank)
                      : plan_adapters_as<DT, false>(adapters, rows, N, K, rank);
}

struct AdapterGradPlan {
    int64_t chunk, slots, rank_tiles, strips[2], workgroups, part_bytes[2], bytes;
};
// Positions a workgroup takes: kChunk, fewer (down to 64) while there are fewer than 512
// workgroups.
inline AdapterGradPlan plan_adapters_wgrad(int64_t adapters, int64_t rows, int64_t N, int64_t K, int64_t rank, bool f32) {
    AdapterGradPlan p = {};
    const int64_t cols = 4 * (f32 ? StreamShape<DT_F32, false>::COLS : StreamShape<DT_F16, false>::COLS);
    p.chunk = kChunk;
    p.slots = rows > 0 ? tiles_and_slots(rows, adapters, kChunk) : 0;
    p.rank_tiles = cdiv(rank, kWgradRank);
    p.strips[0] = cdiv(K, cols);
    p.strips[1] = cdiv(N, cols);
    p.workgroups = (p.strips[0] + p.strips[1]) * p.rank_tiles * p.slots;
    p.part_bytes[0] = round_up(p.slots * rank * K * 4, 16);
    p.part_bytes[1] = p.slots * rank * N * 4;
    p.bytes = p.part_bytes[0] + p.part_bytes[1];
    return p;
}

}  // namespace tg
