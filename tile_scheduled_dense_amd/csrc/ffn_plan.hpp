// ffn_plan.hpp -- which kernels an operator of a feed-forward block takes, their grids and
// their workspace: host arithmetic on sizes and types alone, shared by the launches
// (gated_kernels.hpp, adapters_kernels.hpp) and the C ABI (ffn.hip).
#pragma once

#include <hip/hip_runtime.h>

#include "adapters.hpp"
#include "experts_plan.hpp"

namespace tg {

struct FewPlan {
    bool few;                    // streamed weights; else block tiles
    int waves, splits;
    ProductPlan product;
};

// Waves of a workgroup that splits K (plan_stream).
inline int few_waves(int64_t stages) { return stages >= 16 ? 8 : (stages >= 8 ? 4 : 2); }

// Splits of K over workgroups, of `groups` at work: until there are 512, at least a
// stage for each wave.
inline int few_splits(int64_t groups, int64_t stages, int waves) {
    int s = 1;
    while (groups * s * 2 <= 512 && stages >= (int64_t)waves * s * 2) s *= 2;
    return s;
}

// ---- the gated pair -----------------------------------------------------------------------
template <int DT, bool TRANS>
FewPlan plan_gated(int64_t experts, int64_t rows, int64_t N, int64_t K) {
    using S = StreamShape<DT, TRANS>;
    FewPlan p = {};
    const int64_t mean = cdiv(rows, experts), cols = TwoStrips<DT, TRANS>::COLS;
    const int64_t weights = 2 * experts * N * K * S::E;
    const int64_t strips = cdiv(N, cols) * experts * cdiv(mean, 16);
    p.few = N < kNarrow || (weights <= (int64_t(96) << 20) && (mean <= 8 || (mean <= 128 && strips < 256))) || mean <= 64;
    if (p.few) {
        const int64_t stages = cdiv(K, S::K), used = rows < experts ? rows : experts;
        p.waves = few_waves(stages);
        p.splits = few_splits(cdiv(N, cols) * used * cdiv(cdiv(rows, used), 16), stages, p.waves);
        p.product = plan_of(TG_EXPERTS_STREAM, 16, (int)cols, p.waves, cdiv(N, cols) * p.splits,
                            tiles_and_slots(rows, experts, 16));
        return p;
    }
    const int64_t tiles = cdiv(rows, 256) * cdiv(N, 128);
    if (DT == DT_F32) p.product = plan_tiles(experts, rows, N, 64, 64, false, true, 4);
    else if (K >= kLong && tiles >= 128) p.product = plan_tiles(experts, rows, N, 256, 128, true, true, 4);
    else p.product = plan_tiles(experts, rows, N, 128, 64, false, false, 3);
    return p;
}
template <int DT>
FewPlan plan_gated(bool transposed, int64_t experts, int64_t rows, int64_t N, int64_t K) {
    return transposed ? plan_gated<DT, true>(experts, rows, N, K) : plan_gated<DT, false>(experts, rows, N, K);
}
inline int64_t gated_workspace(const FewPlan &p, int64_t rows, int64_t N) {
    return p.few && p.splits > 1 ? p.splits * 2 * rows * N * 4 : 0;
}

// The gate's gradient: the products' own rule (plan_grouped).

// ---- adapters -------------------------------------------------------------------------------
// At most so many rows are taken by streaming W.
constexpr int64_t kAdapterFew = 64;

struct AdapterPlan {
    bool few;
    int waves, splits;           // x . W
    int t_waves, t_splits;       // x . A[g]
    int64_t ld_low;              // many rows: t's row length
    int64_t part_bytes, bytes;   // workspace: sums of x . W, all
    ProductPlan product;
};

template <int DT, bool TRANS>
AdapterPlan plan_adapters(int64_t adapters, int64_t rows, int64_t N, int64_t K, int64_t rank) {
    using S = StreamShape<DT, TRANS>;
    AdapterPlan p = {};
    const int64_t stages = cdiv(K, S::K);
    p.few = rows <= kAdapterFew || N < kNarrow;
    p.waves = p.t_waves = few_waves(stages);
    p.splits = p.t_splits = 1;
    if (p.few) {
        const int64_t strips = cdiv(N, S::COLS), row_tiles = cdiv(rows, 16);
        p.splits = few_splits(strips * row_tiles, stages, p.waves);
        p.t_splits = few_splits(8, stages, p.waves) < 8 ? few_splits(8, stages, p.waves) : 8;
        p.part_bytes = round_up(p.splits * rows * N * 4, 16);
        p.bytes = p.part_bytes + p.t_splits * rows * rank * 4;
        p.product = plan_of(TG_EXPERTS_STREAM, 16, S::COLS, p.waves, strips * row_tiles * p.splits +
                            cdiv(rank, S::COLS) * p.t_splits * tiles_and_slots(rows, adapters, 16));
        return p;
    }
    p.ld_low = round_up(rank, S::PER);
    p.bytes = rows * p.ld_low * S::E;
    const int64_t tiles = cdiv(rows, 256) * cdiv(N, 256);
    if (DT == DT_F32) p.product = plan_tiles(1, rows, N, 64, 64, false, true, 4);
    else if (K >= kLong && tiles >= 128) p.product = plan_tiles(1, rows, N, 256, 256, true, true, 4);
    else p.product = plan_tiles(1, rows, N, 128, 128, false, false, 3);
    return p;
}
template <int DT>
AdapterPlan plan_adapters(bool transposed, int64_t adapters, int64_t rows, int64_t N, int64_t K, int64_t rank) {
    return transposed ? plan_adapters<DT, true>(adapters, rows, N, K, rank)
                      : plan_adapters<DT, false>(adapters, rows, N, K, rank);
}

struct AdapterGradPlan {
    int64_t slots, rank_tiles, strips[2], workgroups, part_bytes[2], bytes;
};
inline AdapterGradPlan plan_adapters_wgrad(int64_t adapters, int64_t rows, int64_t N, int64_t K, int64_t rank, bool f32) {
    AdapterGradPlan p = {};
    const int64_t cols = 4 * (f32 ? StreamShape<DT_F32, false>::COLS : StreamShape<DT_F16, false>::COLS);
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
