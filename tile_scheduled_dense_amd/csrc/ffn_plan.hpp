// ffn_plan.hpp -- which kernels an operator of a feed-forward block takes, their grids and
// their workspace: host arithmetic on sizes and types alone, shared by the launches
// (gated_kernels.hpp, adapters_kernels.hpp) and the C ABI (ffn.hip).
#pragma once

#include <hip/hip_runtime.h>

#include "adapters.hpp"
#include "experts_plan.hpp"

namespace tg {

// Bytes of a workspace's part, a multiple of 16; kNoMemory where no memory holds them (extents
// up to 2^30 each, so that their product may pass 64 bits).
constexpr int64_t kNoMemory = int64_t(1) << 50;
inline int64_t part_bytes(int64_t copies, int64_t rows, int64_t cols, int64_t element) {
    const unsigned __int128 n = (unsigned __int128)copies * rows * element * cols;
    return n < kNoMemory - 16 ? round_up((int64_t)n, 16) : kNoMemory;
}

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
// Which kernel, by rows of an expert on average, and what the other one takes:
//  * Streamed weights, both strips of a column in a workgroup of up to 8 waves along K: up to
//    16 rows of weights outputs x inputs (8192 x 4096 f16, 16 rows 32.0 us, tiles 37.5; 24 rows
//    52.3 and 38.0; 2816 x 1024, 1 row 8.0 and 11.2) and in fp32 (4096 x 1024, 16 rows 12.7 and
//    18.0; 4096 x 2048, 32 rows 38.7 and 28.7); 16 bits as stored take tiles at once (8192 x
//    4096 f16, 1 row 28.8 us on tiles, 31.6 streamed; 16 rows 30.4 and 38.3).
//  * Tiles of 64 x 64 with K split over workgroups up to 64 rows, in 16 bits up to 128 where
//    the strips are few (one expert of 4096 x 2048, 65 rows 15.9 us against 25.3 on 128 x 64,
//    128 rows 18.5 and 25.0, 256 rows 25.1 and 25.0; 8 experts of 2048 x 1024, 640 rows, 256
//    strips, 23.6 and 19.4; fp32, 640 rows 101 and 65).
//  * Split too for more rows where tiles are few and K is long (at most 128 tiles, fp32 64, of
//    64 K tiles or more; a split 32, fp32 16: 256 rows of 1024 x 4096 bf16 in 1 and 4 splits 34.5 and
//    19.7 us, 512 rows in 1 and 2 36.1 and 28.5, of 512 x 1024 in 1 and 2 11.2 and 12.1; fp32
//    325 rows of 104 x 3320 in 1 and 8 99 and 24, 512 rows of 1024 x 1024, 128 tiles, 34.9 and 40.8).
//  * The same tile, not split, in 16 bits where tiles of 128 x 64 are up to 400 (517 x 1001, 2501
//    rows 24.2 us against 25.8; 1024 x 512 18.1 and 18.9; 8192 rows 49.4 and 45), but not where K
//    is long and tiles are more than the CUs (375 rows of 4208 x 6152 155 and 107; 13462 rows of
//    136 x 4840 150 and 117; 1024 rows of 1024 x 4096, 256 tiles, 41.3 and 42.7).
//  * 256 x 128 with the pipeline where K is long and the tiles fill more than half the card (256
//    tiles, 2048 rows of 4096 x 4096, 104 us, on 128 x 64 164; 128 tiles, 512 rows of 8192 x 4096, 111
//    and 95, 4096 rows of 1024 x 8192 174 and 163, 1024 rows of 4096 x 4096 76.8 and 79.2).
// The splits of K go up to 256 workgroups (48 rows f16, 128, 256, 512, 1024 workgroups: 44.1, 33.8,
// 39.8, 47.0 us; 2816 x 1024, 1 row in 1 split 8.0, in 2 10.9), none shorter than the waves' stages.
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
    const int64_t strips = cdiv(N, 64) * used, k_tiles = cdiv(K, 64 / S::E), all = cdiv(N, 64) * (cdiv(rows, 64) + used - 1);
    const bool split = mean <= 64 || (DT != DT_F32 && mean <= 128 && strips <= 128);
    const bool deep = !split && k_tiles >= 64 && all <= (DT == DT_F32 ? 64 : 128);
    if (split || deep || (DT != DT_F32 && cdiv(rows, 128) * cdiv(N, 64) <= 400 && (K < 2048 || all <= 256))) {
        p.splits = split ? few_splits(strips, 256, k_tiles, 8)
                         : (deep ? few_splits(all, 256, k_tiles, DT == DT_F32 ? 16 : 32) : 1);
        p.product = plan_of(TG_EXPERTS_TILES, 64, 64, 4, cdiv(N, 64) * p.splits, tiles_and_slots(rows, experts, 64));
        return p;
    }
    const int64_t tiles = cdiv(rows, 256) * cdiv(N, 128);
    if (DT == DT_F32) p.product = plan_tiles(experts, rows, N, 64, 64, false, true, 4);
    else if (K >= kLong && tiles > 128) p.product = plan_tiles(experts, rows, N, 256, 128, true, true, 4);
    else p.product = plan_tiles(experts, rows, N, 128, 64, false, false, 3);
    return p;
}
template <int DT>
GatedPlan plan_gated(bool transposed, int64_t experts, int64_t rows, int64_t N, int64_t K) {
    return transposed ? plan_gated_as<DT, true>(experts, rows, N, K) : plan_gated_as<DT, false>(experts, rows, N, K);
}
inline int64_t gated_workspace(const GatedPlan &p, int64_t rows, int64_t N) {
    return p.splits > 1 ? part_bytes(p.splits * 2, rows, N, 4) : 0;
}

// The gate's gradient: the products' own rule (plan_grouped_as), but the smaller tiles of 16
// bits are smaller still, their epilogue reads and writes four matrices: 128 x 128, 64 x 128 and
// 64 x 64 take 32.3, 25.6, 20.8 us (2501 rows of 517 x 1001), 23, 17.7, 14.8 (1024 x 512), 44,
// 37.9, 39.0 (8192 rows); with a long K 64 x 128 and 64 x 64 take 70.6 and 61.8 (2048 rows of 1024 x
// 8192, 256 tiles), 28.4 and 29.7 (1024 of 2816 x 2048, 352), 66 and 90 (512 of 8192 x 4096, 512);
// the large tiles of 256 x 256 stay (16384 rows of 8 experts of 2048 x 2048 210 us, 128 x 128 234,
// 64 x 64 354).  K is not split here, so a long one with few tiles leaves CUs idle (bf16, 100 rows
// of 500 x 8000, streamed, 32 workgroups, 186 us, where the pair itself takes 18 in 16 splits).
template <int DT, bool TRANS>
ProductPlan plan_gate_grad_as(int64_t experts, int64_t rows, int64_t N, int64_t K) {
    const ProductPlan p = plan_grouped_as<DT, TRANS>(experts, rows, N, K);
    if (DT == DT_F32 || p.info.kernel != TG_EXPERTS_TILES || p.info.tile_m == 256) return p;
    return plan_tiles(experts, rows, N, 64, cdiv(rows, 64) * cdiv(N, 128) <= (K < 2048 ? 512 : 300) ? 64 : 128, false, false, 4);
}

template <int DT>
ProductPlan plan_gate_grad(bool transposed, int64_t experts, int64_t rows, int64_t N, int64_t K) {
    return transposed ? plan_gate_grad_as<DT, true>(experts, rows, N, K) : plan_gate_grad_as<DT, false>(experts, rows, N, K);
}

// ---- adapters -------------------------------------------------------------------------------
// Few rows: a projection's columns and its adapters' share one launch, and another adds them
// up.  So up to 64 rows, and up to 512 where that makes at most 192 tiles of 64 x 64; more
// take three launches or four (t, its join, the tiles, their join).  20 adapters of rank 16,
// bf16, few against many: 4096 x 4096, 65 rows 23.6 and 49.6 us, 128 rows 26.2 and 52.1, 192
// rows (192 tiles) 39.1 and 48.3; one adapter, 256 rows (256 tiles) 41.9 and 32.8; 2048 x 8192,
// 256 rows 39.3 and 49.3; 16384 x 4096, 128 rows (512 tiles) 104 and 82; 1024 x 4096,
// 768 rows 43.8 and 37.6; one adapter of rank 64 of 512 x 8192, 1024 rows 54.8 and 37.0; fp32
// 4096 x 4096, 256 rows (256 tiles) 124 and 90; 771 x 1540, 512 rows (104 tiles) 59.7 and 85.0.
// The rank is not looked at, though few rows read its B again for each: 8 adapters of rank 128,
// bf16, as stored and transposed, 65 rows of 4096 x 4096 32.4 and 39.0 us against 61.2 and 56.6 as
// many, 192 rows 51.1 and 78.7 against 55.6 and 52.1; of rank 512, 65 rows 71.2 and 98.7 against 202
// and 177, 192 rows 110 and 228 against 151 and 135; 512 rows of 1536 x 4096, rank 1024, 157 and 95.5.
inline bool adapters_few(int64_t rows, int64_t N) {
    return rows <= 64 || N < kNarrow || (rows <= 512 && cdiv(rows, 64) * cdiv(N, 64) <= 192);
}

enum { ADAPTERS_STREAM = 0, ADAPTERS_SPLIT = 1, ADAPTERS_TILES = 2 };
struct AdapterPlan {
    int form;
    int splits, t_splits;        // of K: x . W, x . A[g]
    int64_t ld_low;              // tiles: t's row length
    int64_t part_bytes, part_t_bytes, bytes;   // workspace: sums of x . W, of x . A[g], all
    ProductPlan product;         // ADAPTERS_STREAM, _SPLIT: without the workgroups of x . A[g]
    ProductPlan low;             // x . A[g]
};

// Few rows: streamed weights up to 16 rows as the gated pair has them (one row of 4096 x 4096,
// 13.1 us; as stored in 16 bits 18.1 on tiles and 18 to 21 streamed), K split up to 512 workgroups
// (128, 256, 512: 17.8, 13.1, 13.1 us, fp32 32.9, 25.9, 19.2) of 4 waves (8 waves 13.7 to 15);
// tiles up to 256 (64 rows, 128, 256, 512: 21.7, 17.0, 18.9 us, as stored 29.9, 24.4, 27.3), t
// in 8 splits (4, 8, 16: 18.6, 17.2, 17.5; as stored 8 and 16 24.5 and 28.7).
// Many: t on tiles of 64 x 64, split up to 512 workgroups (8192 rows, up to 512 252 us, 2048 259);
// the product as the products have it, 256 x 256 in two halves of a very long K too where whole
// ones would leave up to three quarters of the CUs idle (against 128 x 128: 796 rows of 7296 x 6632 135
// and 197 us, 2798 of 1800 x 7568 131 and 165, 1792 of 2560 x 8192 120 and 139, x 4096 74.5 and
// 71.4, 1280 of 4096 x 4096 77.5 and 72.2; 512 of 8704 x 8192, 68 tiles, 128 and 173, of 8192 x 8192,
// 64 tiles, 120 and 112, 1024 of 4096 x 8192, 64, 120 and 115, 2048 of 1536 x 8192, 48, 110 and 84.7;
// 1792 of 2560 x 6144, 70 tiles, 100 and 111, 1024 of 4352 x 6144, 68, 105 and 98, x 5120 92 and 84),
// its smaller tiles split where a half is still 16 tiles of K long (fp32 771 x 1540, 1333 rows, in
// 1, 2, 4 splits: 121, 125, 141 us).
template <int DT, bool TRANS>
AdapterPlan plan_adapters_as(int64_t adapters, int64_t rows, int64_t N, int64_t K, int64_t rank) {
    using S = StreamShape<DT, TRANS>;
    AdapterPlan p = {};
    const int64_t stages = cdiv(K, S::K), k_tiles = cdiv(K, 64 / S::E);
    p.splits = p.t_splits = 1;
    if (adapters_few(rows, N)) {
        const bool stream = N < kNarrow || (rows <= 16 && (TRANS || DT == DT_F32));
        const int waves = 4;
        p.form = stream ? ADAPTERS_STREAM : ADAPTERS_SPLIT;
        const int64_t strips = cdiv(N, stream ? S::COLS : 64), tiles = strips * cdiv(rows, stream ? 16 : 64);
        p.splits = stream ? few_splits(tiles, 512, stages, waves) : few_splits(tiles, 256, k_tiles, 8);
        p.t_splits = few_splits(cdiv(rank, S::COLS), 8, stages, waves);
        p.part_bytes = part_bytes(p.splits, rows, N, 4);
        p.part_t_bytes = part_bytes(p.t_splits, rows, rank, 4);
        p.product = plan_of(stream ? TG_EXPERTS_STREAM : TG_EXPERTS_TILES, stream ? 16 : 64, stream ? S::COLS : 64, waves,
                            tiles * p.splits);
        p.low = plan_of(TG_EXPERTS_STREAM, 16, S::COLS, waves,
                        cdiv(rank, S::COLS) * p.t_splits * tiles_and_slots(rows, adapters, 16));
    } else {
        p.form = ADAPTERS_TILES;
        p.ld_low = round_up(rank, S::PER);
        p.t_splits = few_splits(cdiv(rows, 64) * cdiv(rank, 64), 512, k_tiles, 8);
        p.part_t_bytes = part_bytes(p.t_splits, rows, rank, 4);
        p.low = plan_of(TG_EXPERTS_TILES, 64, 64, 4, cdiv(rank, 64) * p.t_splits, tiles_and_slots(rows, adapters, 64));
        const int64_t tiles = cdiv(rows, 256) * cdiv(N, 256);
        if (DT == DT_F32) p.product = plan_tiles(1, rows, N, 64, 64, false, true, 4);
        else if (K >= kLong && tiles >= 128) p.product = plan_tiles(1, rows, N, 256, 256, true, true, 4);
        else if (K >= 6144 && tiles > 64) p.product = plan_tiles(1, rows, N, 256, 256, false, true, 4), p.splits = 2;
        else p.product = plan_tiles(1, rows, N, 128, 128, false, false, 3);
        if (p.splits > 1 || p.product.info.tile_m < 256) {
            if (p.splits == 1) p.splits = few_splits(p.product.gx, 512, k_tiles, 16);
            if (p.splits > 1) p.part_bytes = part_bytes(p.splits, rows, N, 4);
            const bool pipeline = p.product.info.pipeline;
            p.product = plan_of(TG_EXPERTS_TILES, p.product.info.tile_m, p.product.info.tile_n, 4, p.product.gx * p.splits);
            p.product.info.pipeline = pipeline;
        }
    }
    p.bytes = p.part_bytes + p.part_t_bytes + part_bytes(1, rows, p.ld_low, S::E);
    return p;
}
template <int DT>
AdapterPlan plan_adapters(bool transposed, int64_t adapters, int64_t rows, int64_t N, int64_t K, int64_t rank) {
    return transposed ? plan_adapters_as<DT, true>(adapters, rows, N, K, rank)
                      : plan_adapters_as<DT, false>(adapters, rows, N, K, rank);
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
    // an adapter's chunks are added up where it has several
    const int64_t places = rows > kChunk ? 2 * cdiv(rows, kChunk) : 0;
    p.part_bytes[0] = part_bytes(places, rank, K, 4);
    p.part_bytes[1] = part_bytes(places, rank, N, 4);
    p.bytes = p.part_bytes[0] + p.part_bytes[1];
    return p;
}

}  // namespace tg
