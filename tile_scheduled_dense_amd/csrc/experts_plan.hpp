// experts_plan.hpp -- which kernel an expert product takes and the grid it is
// started with: host arithmetic on sizes and types alone, shared by the launches
// (experts_kernels.hpp) and the plan queries of the C ABI (experts.hip).
#pragma once

#include <hip/hip_runtime.h>

#include "experts.hpp"
#include "grid.hpp"
#include "ranges.hpp"
#include "tile_gemm_experts.h"

namespace tg {

struct ProductPlan {
    tg_experts_plan_info info;
    int lds_copies;              // of a K tile (tiles)
    int64_t gx;                  // workgroups: gx * gy * gz
    unsigned gy, gz;
    bool fits() const { return grid_fits(gx, 64 * info.waves); }
};

inline ProductPlan plan_of(int kernel, int tile_m, int tile_n, int waves, int64_t gx, int64_t gy = 1, int64_t gz = 1) {
    ProductPlan p = {};
    p.info.kernel = kernel;
    p.info.tile_m = tile_m;
    p.info.tile_n = tile_n;
    p.info.waves = waves;
    p.info.workgroups = gx * gy * gz;
    p.info.row_tiles = 1;
    p.gx = gx;
    if (gy > kGridY) {                    // in whole layers (slot_of)
        gz = cdiv(gy, kGridY);
        gy = kGridY;
    }
    p.gy = (unsigned)gy;
    p.gz = (unsigned)gz;
    return p;
}

// Waves that split K: enough for two stages each, eight at most.
template <int DT, bool TRANS>
ProductPlan plan_stream(int64_t experts, int64_t rows, int64_t N, int64_t K) {
    using S = StreamShape<DT, TRANS>;
    const int64_t stages = cdiv(K, S::K);
    const int waves = stages >= 16 ? 8 : (stages >= 8 ? 4 : 2);
    return plan_of(TG_EXPERTS_STREAM, 16, S::COLS, waves, cdiv(N, S::COLS), tiles_and_slots(rows, experts, 16));
}

// the most tile rows that `groups` groups of `rows` rows together can have
inline int64_t most_tiles(int64_t rows, int64_t groups, int64_t bm) {
    const int64_t parts = rows < groups ? rows : groups;
    return (rows + parts * (bm - 1)) / bm;
}

// The grid is the most there can be: whole tiles and, with pieces, three more for each
// tile that is split, and a row of pieces for every group.
inline ProductPlan plan_tiles(int64_t experts, int64_t rows, int64_t N, int tile_m, int tile_n, bool pieces, bool pipeline,
                              int copies) {
    int64_t grid = most_tiles(rows, experts + 1, tile_m) * cdiv(N, tile_n);
    if (pieces) grid += 3 * kSplitRound + (rows < experts + 1 ? rows : experts + 1) * cdiv(N, tile_n / 2);
    ProductPlan p = plan_of(TG_EXPERTS_TILES, tile_m, tile_n, 4, grid);
    p.info.pieces = pieces;
    p.info.pipeline = pipeline;
    p.lds_copies = copies;
    return p;
}

// A contraction long enough that the 256 x 256 tile's rate outweighs what its start
// and its stores cost, which the two or three workgroups of 128 x 128 that a CU holds
// hide in each other (bf16, 8 uneven experts: 16384 x 4096 over K 256 55 us on 128 x 128
// against 70, 512 86 against 96, 8192 x 4096 over 1024 81 against 78; the weights'
// gradient of 2048 x 2048 over 512 rows an expert 86 against 99, over 1024 75 against 74).
constexpr int64_t kLong = 1024;

// The tile of a product over rows.
//  * The weights are streamed, by workgroups that split K among their waves, while they
//    are at most 96 MiB and an expert has on average at most 8 rows, or at most 128 in
//    fewer than 256 workgroups.  bf16, streamed and on tiles, weights from HBM:
//      up to 8 rows    8 experts of 1024 x 4096 (K x N), 32 rows 16.3 and 19.5 us; one of
//                      1024 x 4096, 8 rows 7.6 and 14.5
//      16 each         8 of 2048 x 4096, even 29.7 and 32.5, skewed 38.3 and 32.4
//      workgroups      16 of 512 x 256, 63 rows each, 128 of them, 6.9 and 9.4, 125 rows, 256,
//                      11.3 and 9.7; 2 of 2048 x 4096 transposed, 128 rows each, 2048, 49.5
//                      and 29.3
//      96 MiB          12 of 1024 x 4096, 48 rows 26.3 and 22.9, 64 of 1024 x 768, 512 rows
//                      skewed 25.6 and 31.7; more: 64 of 2048 x 2048, 500 rows 101 and 114
//                      (transposed 92 and 115), but in one expert 28.7 and 25.5 (50 and 24)
//    So is an N below kNarrow, of which a tile would be mostly empty (and the tiles need a
//    16-byte chunk of it: grouped_ring.hpp).
//  * 16 bits: 256 x 256 over a long K from 128 such tiles on (f16, 8 uneven experts, K
//    1024: 4096 x 2048 32.0 against 33.4 us on 128 x 128, 2048 x 2048 26.5 against 22.6),
//    else 128 x 128, three LDS copies for three workgroups a CU (257 x 1000 over 150 rows
//    18.9 us with four copies, 17.0 with three, 16.8 with two, which cost 5001 x 257 over
//    1000 28.4 against 21.9).
//  * fp32: 64 x 64, more workgroups for a matrix rate that 16 of them already fill
//    (2048 x 1024 x 512 30 us against 42 on 128 x 128; 4096 x 4096 x 512 149, 173 and 163
//    on 256 x 256), with the software pipeline (2048 x 1024 x 512 28 us, 30 without);
//    256 x 256 from 800 tiles on (16384 x 4096 x 2048 1979 against 2147).
template <int DT, bool TRANS>
ProductPlan plan_grouped_as(int64_t experts, int64_t rows, int64_t N, int64_t K) {
    const int64_t mean = cdiv(rows, experts);
    const int64_t weights = experts * N * K * (DT == DT_F32 ? 4 : 2);
    const int64_t strips = cdiv(N, StreamShape<DT, TRANS>::COLS) * experts * cdiv(mean, 16);
    const bool stream = weights <= (int64_t(96) << 20) && (mean <= 8 || (mean <= 128 && strips < 256));
    if (stream || N < kNarrow) return plan_stream<DT, TRANS>(experts, rows, N, K);
    const int64_t tiles = cdiv(rows, 256) * cdiv(N, 256);
    if (K >= kLong && tiles >= (DT == DT_F32 ? 800 : 128)) return plan_tiles(experts, rows, N, 256, 256, true, true, 4);
    return DT == DT_F32 ? plan_tiles(experts, rows, N, 64, 64, false, true, 4)
                        : plan_tiles(experts, rows, N, 128, 128, false, false, 3);
}
template <int DT>
ProductPlan plan_grouped(bool transposed, int64_t experts, int64_t rows, int64_t N, int64_t K) {
    return transposed ? plan_grouped_as<DT, true>(experts, rows, N, K) : plan_grouped_as<DT, false>(experts, rows, N, K);
}

// The tile of the weights' gradient; its contraction is an expert's rows, on average.
//  * 256 x 256 over a long one from 200 such tiles on, fp32 800 (fewer leave a popular
//    expert's tiles to end alone: 12 uneven experts of 1024 x 1024, 192 tiles, 79 us and 60.5
//    on 128 x 128, even ones 35.5 and 43), where whole rounds of 256 of them (one a CU)
//    cover at most half more than the small tiles do, padding and part-filled rounds
//    together; fp32, whose small tile reaches the same rate, a twentieth more (bf16, 1100
//    rows an expert, 256 x 256 and 128 x 128: 16 experts of 1024 x 1024, a whole round, 44.6
//    and 56.5 us, 20, 1.6, 76.4 and 67.8, 17, 1.88, 74.6 and 62.2; 8 of 1300 x 1304, 2.1, 61
//    and 49; 64 of 512 x 512, 1.0, 54.6 and 71.3; over 2500 rows 1.6 is 133 and 144, 2.1 114
//    and 112; fp32 against 64 x 64: 8 of 2048 x 2048, 1.0, 536 and 545, 4 of 3600 x 3840,
//    1.2, 1385 and 1206).
//  * else 128 x 128, fp32 64 x 64; with the software pipeline where no CU has a second tile
//    to hide the first one's waits (464 x 96 over 1464 rows, 2 experts: 20.4 -> 13.1 us; 33
//    of 257 x 1000 over 150 16.9 -> 20.9).
template <int DT>
ProductPlan plan_wgrad(int64_t experts, int64_t rows, int64_t M, int64_t N) {
    if (M < kNarrow || N < kNarrow) {
        const int width = narrow_width(M < N ? N : M, DT == DT_F32);
        return plan_of(TG_EXPERTS_NARROW, M < N ? (int)M : width, M < N ? width : (int)N, 16, cdiv(M < N ? N : M, width),
                       experts);
    }
    int tile = DT == DT_F32 ? 64 : 128;
    const int64_t small = experts * cdiv(M, tile) * cdiv(N, tile);
    const int64_t large = experts * cdiv(M, 256) * cdiv(N, 256), area = cdiv(large, kRound) * kRound;
    bool pipeline = DT == DT_F32 || small <= 256;
    if (cdiv(rows, experts) >= kLong && (DT == DT_F32 ? large >= 800 && 20 * 16 * area <= 21 * small
                                                      : large >= 200 && 2 * 4 * area <= 3 * small)) {
        tile = 256;
        pipeline = true;
    }
    ProductPlan p = plan_of(TG_EXPERTS_TILES, tile, tile, 4, experts * cdiv(M, tile) * cdiv(N, tile));
    p.info.pipeline = pipeline;
    p.lds_copies = pipeline ? 4 : 3;
    return p;
}

// Column tiles of 16 that a workgroup takes: two, which read the activations once, from 512
// column tiles on, or from 768 tiles with the rows there are on average; below, one, in
// twice the workgroups (one and two, K 4096, bf16: 4096 columns, 16 rows 5.5 and 6.8 us, 32
// rows 7.4 and 9.2, 48 rows 10.3 and 9.3, 64 rows 12.2 and 9.4; 8192, 32 rows 12.9 and 10.1;
// f16: 6144, 16 rows 7.3 and 6.6, 8192 x 8192, 8 rows 9.1 and 9.6, 16 rows 11.7 and 10.6; 64
// experts of 2048 x 2048 with 16 rows each 51.7 and 40.7, 8 with 2 each 6.8 and 7.4).  fp32
// one: 37 rows of 1001 x 4100 11.7 and 17.4, 64 experts of 1024 x 1024 29.6 and 34.6; two pay
// for a large matrix alone (16 rows of 8192 x 8192 33.4 and 28.9).
template <int DT>
ProductPlan plan_q4(int64_t experts, int64_t rows, int64_t N, int64_t K) {
    const int64_t n_tiles = cdiv(N, kQ4N), k_blocks = cdiv(K, kQ4K), all = n_tiles * experts;
    const int nt = DT != DT_F32 && (all >= 512 || all * cdiv(cdiv(rows, experts), 16) >= 768) ? 2 : 1;
    // waves that split K: more while they have four blocks each and there are not yet
    // 4096 (a wave costs 0.6 ns to start: 64 experts of 2048 x 2048, 64 rows, take 24 us in
    // workgroups of 1 wave, 15.5 of 2, 16.4 of 4, 20 of 8; one of 4096 x 4096, 16 rows, 16,
    // 9.5, 6.7 and 5.5)
    const int64_t strips = cdiv(n_tiles, nt);
    int waves = 1;
    while (waves < q4_waves<DT>() && waves * 4 <= k_blocks && (waves < 2 || strips * experts * waves < 4096)) waves *= 2;
    return plan_of(TG_EXPERTS_Q4, 16, 16 * nt, waves, strips, tiles_and_slots(rows, experts, 16));
}

}  // namespace tg
