// experts_kernels.hpp -- instantiations and launches of the expert products'
// kernels (experts.hpp), included by one translation unit per input type.
#pragma once

#include <hip/hip_runtime.h>

#include "experts.hpp"
#include "ranges.hpp"

namespace tg {
namespace {

inline tg_status launched() { return hipGetLastError() == hipSuccess ? TG_OK : TG_ERR_LAUNCH; }

// Waves that split K: enough for two stages each, eight at most.
template <int DT, bool TRANS>
tg_status launch_stream(const GroupedParams &p, hipStream_t s) {
    using S = StreamShape<DT, TRANS>;
    const int64_t stages = cdiv(p.K, S::K);
    const int waves = stages >= 16 ? 8 : (stages >= 8 ? 4 : 2);
    // Row tiles at the same time: all there can be, if one expert had every row, while
    // that is two workgroups a CU at most; else twice an expert's on average.
    const int64_t strips = cdiv(p.N, S::COLS), mean = cdiv(2 * cdiv(p.rows, p.experts), 16);
    int64_t tiles = cdiv(p.rows, 16) < 8 ? cdiv(p.rows, 16) : 8;
    while (tiles > 1 && tiles > mean && strips * (p.experts + 1) * tiles > 512) --tiles;
    const dim3 grid((unsigned)strips, (unsigned)p.experts + 1, (unsigned)tiles);
    hipLaunchKernelGGL((grouped_stream_kernel<DT, TRANS>), grid, dim3(64 * waves), waves * S::FRAGS * 1024, s, p);
    return launched();
}

template <int DT, int GROUP, int MT, int NT>
tg_status launch_q4_as(const Q4Params &p, int64_t chunks, hipStream_t s) {
    // waves that split K: more while they have four blocks each and there are not yet
    // 4096 (a wave costs 0.6 ns to start: 64 experts of 2048 x 2048, 24 of them with
    // rows, take 15 us in workgroups of 2 waves, 17 of 4, 27 of 8)
    const int64_t strips = cdiv(p.n_tiles, NT);
    int waves = 1;
    while (waves < q4_waves<DT, MT>() && waves * 4 <= p.k_blocks && (waves < 2 || strips * p.experts * waves < 4096))
        waves *= 2;
    const unsigned lds = waves * Q4Rows<DT, MT>::LDS * 16;
    const dim3 grid((unsigned)strips, (unsigned)p.experts + 1, (unsigned)cdiv(chunks, MT));
    hipLaunchKernelGGL((q4_kernel<DT, GROUP, MT, NT>), grid, dim3(64 * waves), lds, s, p);
    return launched();
}

// Row tiles (MT) and n tiles (NT) of a workgroup: more of either reads the codes or
// the activations less often, as long as there are workgroups for the 256 CUs.
// fp32 takes one of each, in as many workgroups: two row tiles leave room for half the
// waves, whose latency then shows (37 rows, 1001 x 4100: 12 us against 28).
// chunks: row tiles that an expert has on average.
template <int DT, int GROUP>
tg_status launch_q4_group(const Q4Params &p, hipStream_t s) {
    const int64_t chunks = cdiv(cdiv(p.rows, p.experts), 16) < 64 ? cdiv(cdiv(p.rows, p.experts), 16) : 64;
    const int64_t strips = (int64_t)p.n_tiles * p.experts;
    if constexpr (DT == DT_F32) {
        return launch_q4_as<DT, GROUP, 1, 1>(p, chunks, s);
    } else {
        if (chunks > 2 && strips * cdiv(chunks, 4) >= 256) return launch_q4_as<DT, GROUP, 4, 1>(p, chunks, s);
        if (chunks > 1 && strips * cdiv(chunks, 2) >= 256) return launch_q4_as<DT, GROUP, 2, 1>(p, chunks, s);
        if (strips * chunks >= 512) return launch_q4_as<DT, GROUP, 1, 2>(p, chunks, s);
        return launch_q4_as<DT, GROUP, 1, 1>(p, chunks, s);
    }
}

template <int DT> using Tile256 = RingCfg<DT, 256, 256, 2, 2, 16>;
template <int DT> using Tile128 = RingCfg<DT, 128, 128, 2, 2, 16>;
using Tile64F32 = RingCfg<DT_F32, 64, 64, 2, 2, 16>;

// the most tile rows that `groups` groups of `rows` rows together can have
inline int64_t most_tiles(int64_t rows, int64_t groups, int64_t bm) {
    const int64_t parts = rows < groups ? rows : groups;
    return (rows + parts * (bm - 1)) / bm;
}

// P: the pieces' configuration (C itself: none).  The grid is the most there can
// be: whole tiles, three more pieces for each tile that is split, and a row of
// pieces for every group.
template <class C, class P, bool B_KS, bool PIPE, int STAGES = 4>
tg_status launch_tiles(const GroupedParams &p, hipStream_t s) {
    int64_t grid = most_tiles(p.rows, p.experts + 1, C::BM) * cdiv(p.N, C::BN);
    if (!std::is_same<C, P>::value)
        grid += 3 * kSplitRound + (p.rows < p.experts + 1 ? p.rows : p.experts + 1) * cdiv(p.N, P::BN);
    if (grid > 0x7fffffffLL) return TG_ERR_UNSUPPORTED;
    hipLaunchKernelGGL((grouped_tile_kernel<C, P, B_KS, PIPE, STAGES>), dim3((unsigned)grid), dim3(C::THREADS), 0, s, p);
    return launched();
}

template <class C, bool PIPE, int STAGES = 4>
tg_status launch_wgrad_tiles(const GroupedParams &p, hipStream_t s) {
    const int64_t tiles = cdiv(p.M, C::BM) * cdiv(p.N, C::BN), grid = p.experts * cdiv(tiles, 8) * 8;
    if (grid > 0x7fffffffLL) return TG_ERR_UNSUPPORTED;
    hipLaunchKernelGGL((wgrad_tile_kernel<C, PIPE, STAGES>), dim3((unsigned)grid), dim3(C::THREADS), 0, s, p);
    return launched();
}

// A contraction long enough that the 256 x 256 tile's rate outweighs what its start
// and its stores cost, which the two or three workgroups of 128 x 128 that a CU holds
// hide in each other (bf16, 8 uneven experts: 16384 x 4096 over K 256 55 us on 128 x 128
// against 70, 512 86 against 96, 8192 x 4096 over 1024 81 against 78; the weights'
// gradient of 2048 x 2048 over 512 rows an expert 86 against 99, over 1024 75 against 74).
constexpr int64_t kLong = 1024;

// The tile of a product over rows.
//  * The weights are streamed, by workgroups that split K among their waves, while they
//    are at most 96 MiB and an expert has on average at most 8 rows, or at most 128 and
//    a workgroup a CU takes all 16-row tiles at the same time (bf16: 8 experts of 1024 x
//    4096, 4 rows 13.6 us against 17.6 on tiles; one of 4096 x 256, 16 rows 14.5 against
//    45.6, 96 rows 14.6 against 45.9; 4 of 2048 x 2048, 24 rows 11.1 against 24.3; but 32
//    of 2048 x 1024, 4 rows, 31.5 against 24.6, where the tiles' copies read at 5.5 TB/s,
//    and two workgroups a CU, 8 experts of 1024 x 4096, 32 rows, 28.7 against 18.1).  So
//    is an N below a chunk, which is not for the tiles (grouped_ring.hpp).
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
tg_status launch_grouped_as(const GroupedParams &p, hipStream_t s) {
    const int64_t mean = cdiv(p.rows, p.experts);
    const int64_t weights = (int64_t)p.experts * p.N * p.K * (DT == DT_F32 ? 4 : 2);
    const int64_t strips = cdiv(p.N, StreamShape<DT, TRANS>::COLS) * p.experts * cdiv(mean, 16);
    const bool stream = weights <= (int64_t(96) << 20) && (mean <= 8 || (mean <= 128 && strips < 256));
    if (!stream && p.N >= 8) {
        const int64_t tiles = cdiv(p.rows, 256) * cdiv(p.N, 256);
        if (p.K >= kLong && tiles >= (DT == DT_F32 ? 800 : 128))
            return launch_tiles<Tile256<DT>, Tile128<DT>, !TRANS, true>(p, s);
        if constexpr (DT == DT_F32) return launch_tiles<Tile64F32, Tile64F32, !TRANS, true>(p, s);
        else return launch_tiles<Tile128<DT>, Tile128<DT>, !TRANS, false, 3>(p, s);
    }
    return launch_stream<DT, TRANS>(p, s);
}

}  // namespace

template <int DT>
tg_status launch_grouped(const GroupedParams &p, bool transposed, hipStream_t s) {
    return transposed ? launch_grouped_as<DT, true>(p, s) : launch_grouped_as<DT, false>(p, s);
}

// The tile of the weights' gradient, by the same rules; its contraction is an expert's
// rows, on average.  256 x 256 from 200 tiles on (16 experts of 1024 x 1024: 29.8 us
// against 32.2 on 128 x 128; 8 experts 35.9 against 32.1), unless 128 x 128 pads the
// extents by a fifth less.  128 x 128 with the software pipeline where no CU has a
// second tile to hide the first one's waits (464 x 96 over 1464 rows, 2 experts: 20.4 ->
// 13.1 us; 33 of 257 x 1000 over 150 16.9 -> 20.9).
template <int DT>
tg_status launch_wgrad(const GroupedParams &p, hipStream_t s) {
    if (p.M >= 8 && p.N >= 8) {
        const int64_t each = cdiv(p.M, 256) * cdiv(p.N, 256), small = cdiv(p.M, 128) * cdiv(p.N, 128);
        if (p.experts * each >= (DT == DT_F32 ? 800 : 200) && 4 * each * 4 <= 5 * small && cdiv(p.rows, p.experts) >= kLong)
            return launch_wgrad_tiles<Tile256<DT>, true>(p, s);
        if constexpr (DT == DT_F32) return launch_wgrad_tiles<Tile64F32, true>(p, s);
        else if (p.experts * small <= 256) return launch_wgrad_tiles<Tile128<DT>, true>(p, s);
        else return launch_wgrad_tiles<Tile128<DT>, false, 3>(p, s);
    }
    const int64_t blocks = cdiv((int64_t)p.experts * p.M * p.N, 256);
    hipLaunchKernelGGL((wgrad_small_kernel<DT>), dim3((unsigned)(blocks < 65536 ? blocks : 65536)), dim3(256), 0, s, p);
    return launched();
}

template <int DT>
tg_status launch_q4(const Q4Params &p, int group, hipStream_t s) {
    switch (group) {
        case 32: return launch_q4_group<DT, 32>(p, s);
        case 64: return launch_q4_group<DT, 64>(p, s);
        case 128: return launch_q4_group<DT, 128>(p, s);
    }
    return TG_ERR_INTERNAL;
}

}  // namespace tg
