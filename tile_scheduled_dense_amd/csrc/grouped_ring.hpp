// grouped_ring.hpp -- expert products with many rows an expert, and their
// gradients, on block tiles and the LDS ring of gemm_ring.hpp: one workgroup a
// tile of one expert, K tiles copied straight from memory to LDS a few ahead,
// one barrier per K tile, 16x16x32 (fp32: 16x16x4) matrix instructions.
//
// Three forms, by which axis each operand holds contiguous:
//   C[r] = A[r] . B[g]             A along k,  B along n   (NN)
//   C[r] = A[r] . B[g]^T           both along k            (NT)
//   C[g] = A[rows]^T . D[rows]     A along m, D along n; k is the expert's rows  (TN)
// An operand contiguous along k is staged as rows of 64 bytes and read by
// ds_read_b128; one contiguous along its own extent as 32 k rows and read by
// the transposing ds_read_b64_tr_b16 (fp32: ds_read_b32 per step): the two
// staged tiles of tile_config.hpp, either of them for either operand.
//
// The extents' fringe: a row or column chunk past the end is fetched from past
// the resource, which reads 0.  A chunk that the end cuts brings what lies
// behind, in the same matrix (the host keeps extents below one chunk away; for an
// adapter's rank narrow.hpp), and only feeds outputs that are not stored.  A last K
// tile that K cuts (or whose last chunk would pass a matrix's end) goes through
// registers with element-exact zeros in both operands, so that a NaN behind K meets none.
//
// Measured, 16384 rows x 4096 x 2048 bf16 over 8 experts with a bf16 result, inputs that
// change from call to call: even experts 229 us forward, 229 for the rows' gradient, 219 for
// the weights' (1200-1255 TFLOP/s); uneven ones 240-245, 259-267 and 219-223, where
// part-filled tile rows and the last round show.  On the same inputs again, half of them in
// the last-level cache, 214, 207 and 208 (1282-1329 TFLOP/s, the rate of a large library
// product on this card) and 227, 234 and 211.  Bound by the matrix cores while K is long;
// under about 1024 by the start and the stores of a tile.
//
// B's fragments are the matrix instruction's first operand and A's the second:
// a lane then holds four neighbouring columns of one row of C, so that C is
// stored 8 or 16 bytes at a time.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gemm_ring.hpp"
#include "grouped_stream.hpp"

namespace tg {

template <class C> struct SwapCfg;
template <int DT, int BM, int BN, int WM, int WN, int MT>
struct SwapCfg<RingCfg<DT, BM, BN, WM, WN, MT>> {
    using type = RingCfg<DT, BN, BM, WN, WM, MT>;
};

// One operand of a tile.  V: a configuration whose A tile (contiguous along k)
// or B tile (KS: along the extent) is this operand's.  T: its MFMA tiles per wave.
template <class V, bool KS, int T>
struct RingOperand {
    using CP = RingCopy<V, SWZ_XOR, KS ? 1 : 0>;
    static constexpr int E = V::ELEM, CHUNK = V::CHUNK, BK = V::BK, PER = CP::PER, REGION = CP::REGION;
    static constexpr int SHIFT = (CP::GMAX - 1) * 1024;      // a group's resource base sits this far below
    static constexpr int BASES = KS ? T : 1;                 // registers of fragment read addresses
    static constexpr int PIECES = KS ? (V::DT == DT_F32 ? 4 : 2) : 1;
    // a fragment's largest distance from its base: the last row tile, the last piece
    static constexpr int REACH = KS ? 4 * V::B_ROW_BYTES : (T - 1) * 16 * V::A_ROW_BYTES;
    static_assert(V::MT == 16 && V::KSTEPS == 1, "one fragment read step per K tile");

    const char *base;
    int ld, left;               // left: rows or columns from the tile's first to the extent's end
    int lane, wave;
    uint32_t lds;
    int x[PER], k[PER], voff[PER];
    uint32_t rd[BASES];
    i32x4 rs;
    uint64_t step;              // bytes per K tile

    // base: the tile's first element; w: the wave's first row or column in the tile
    __device__ __forceinline__ void init(const char *base_, int64_t ld_, int left_, int w, uint32_t lds_, int lane_,
                                         int wave_) {
        base = reinterpret_cast<const char *>(uniform_u64(reinterpret_cast<uint64_t>(base_)));
        ld = (int)ld_;
        left = left_;
        lane = lane_;
        wave = wave_;
        lds = lds_;
        step = (uint64_t)(KS ? BK * ld_ * E : BK * E);
        rs = rsrc_words_u(reinterpret_cast<uint64_t>(base) - SHIFT, 0x7fffffff);
#pragma unroll
        for (int d = 0; d < PER; ++d) {
            if constexpr (KS) ring_b_source<V>(CP::block(d, wave), lane, SWZ_XOR, k[d], x[d]);
            else ring_a_source<V>(CP::block(d, wave), lane, SWZ_XOR, x[d], k[d]);
            const int off = x[d] < left ? (KS ? k[d] * ld + x[d] : x[d] * ld + k[d]) * E : kOutOfRange;
            voff[d] = off + SHIFT - 1024 * CP::pos(d);
        }
        const int grp = lane / 16, in = lane % 16;
#pragma unroll
        for (int j = 0; j < BASES; ++j) {
            if constexpr (!KS) rd[j] = lds + ring_a_byte<V>(w + in, grp, SWZ_XOR);
            else if constexpr (V::DT == DT_F32) rd[j] = lds + ring_b_byte<V>(4 * grp, w + 16 * j + in, SWZ_XOR);
            else rd[j] = lds + ring_b_byte<V>(8 * grp + in / 4, w + 16 * j + 4 * (in % 4), SWZ_XOR);
            // keeps the base whole: a split-off constant would not fit the DS offset
            asm("" : "+v"(rd[j]));
        }
    }

    // this wave's copies of the next K tile into LDS copy `stage`
    __device__ __forceinline__ void copy(int stage) {
        constexpr int G0 = CP::Q < 4 ? CP::Q : 4;
        static_assert(CP::Q <= 4 && !CP::SHARED, "one group of copies per wave");
        copy_group_to_lds<G0>(rs, lds + stage * REGION + CP::block(0, wave) * 1024, &voff[0]);
        const uint64_t a = (((uint64_t)(uint32_t)rs.y << 32) | (uint32_t)rs.x) + step;
        rs.x = (int)(uint32_t)a;
        rs.y = (int)(uint32_t)(a >> 32);
    }

    // the K tile at k0, of which k < K exist, through registers, zeros past the ends
    __device__ __forceinline__ void tail_load(int64_t k0, int K, u32x4 *tail) const {
        const rsrc_t r = make_rsrc(base + (KS ? k0 * ld : k0) * E);
#pragma unroll
        for (int d = 0; d < PER; ++d) {
            const int k_left = K - (int)k0 - k[d], x_left = left - x[d];
            const int run = KS ? x_left : k_left, other = KS ? k_left : x_left;
            const int n = other <= 0 || run <= 0 ? 0 : (run < CHUNK ? run : CHUNK);
            tail[d] = bload16_n<E>(r, n > 0 ? (KS ? k[d] * ld + x[d] : x[d] * ld + k[d]) * E : 0, 0, n);
        }
    }
    __device__ __forceinline__ void tail_store(int stage, const u32x4 *tail) const {
#pragma unroll
        for (int d = 0; d < PER; ++d) {
            const uint32_t at = lds + stage * REGION + CP::block(d, wave) * 1024 + 16 * lane;
            *(__attribute__((address_space(3))) u32x4 *)(uintptr_t)at = tail[d];
        }
    }

    // piece q of fragment i from LDS copy `stage`
    __device__ __forceinline__ void read(int stage, int i, int q, u32x4 &f) const {
        if constexpr (!KS) {
            const uint32_t at = rd[0] + stage * REGION + i * 16 * V::A_ROW_BYTES;
            f = *(const __attribute__((address_space(3))) u32x4 *)(uintptr_t)at;
        } else if constexpr (V::DT == DT_F32) {
            const uint32_t at = rd[i] + stage * REGION + q * V::B_ROW_BYTES;
            f[q] = *(const __attribute__((address_space(3))) uint32_t *)(uintptr_t)at;
        } else {
            const uint32_t at = rd[i] + stage * REGION + q * 4 * V::B_ROW_BYTES;
            const u32x2 v = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                                                          (__attribute__((address_space(3))) v4i16 *)(uintptr_t)at));
            if (q == 0) {
                f.x = v.x;
                f.y = v.y;
            } else {
                f.z = v.x;
                f.w = v.y;
            }
        }
    }
};

// Row p of a table of rows, clamped to the rows there are; an entry may be complemented
// (as the token exchange's tables are, for rows without an expert).
__device__ __forceinline__ int row_in(const int32_t *order, int p, int rows) {
    const int r = order[p], t = r < 0 ? ~r : r;
    return t < rows ? t : rows - 1;
}

// The store of a workgroup's tile of a result whose value v (0 .. 3: neighbouring columns)
// of MFMA tile (i, j) of this lane is value(i, j, v) (integral constants).  C: the
// configuration of the product; TN: column tiles of 16 a wave has of the result.
// ORDERED: row m of the tile is row order[m] of C (of `total`), and `at` an offset in a row.
template <class C, int TN, class F, bool ORDERED = false>
struct TileStore {
    const F &value;
    const int lane, wave;
    const int32_t *order = nullptr;
    const int total = 0;
    static constexpr int WTN = 16 * TN, BN = C::WAVES_N * WTN;

    template <int i, int j, int v>
    __device__ __forceinline__ float get() const {
        return value(std::integral_constant<int, i>{}, std::integral_constant<int, j>{}, std::integral_constant<int, v>{});
    }
    // Rows of whole 16-byte units take straight-line code (a tile at an end of C a mask a
    // store), that writes 128 bytes of each of eight rows at a time, whole cache lines
    // where C's rows are aligned to them (64 or 32 bytes a row cost up to 40% more).  Of a
    // 16-bit C a lane holds 8 bytes of each fragment, so neighbouring fragments trade
    // halves between lane groups first (v_permlane16_swap: the odd rows of 16 lanes of
    // one register against the even ones of the other).  Then two 64-byte neighbours P,
    // Q of 16 rows trade their halves of 8 rows (a rotation by 8 lanes).
    __device__ __forceinline__ static void trade_rows(const u32x4 &P, const u32x4 &Q, u32x4 &low, u32x4 &high) {
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            // row_ror:8, written to lanes 8-15 (banks 2, 3) or 0-7 (banks 0, 1) of each 16
            low[c] = __builtin_amdgcn_update_dpp((int)P[c], (int)Q[c], 0x128, 0xf, 0xc, false);
            high[c] = __builtin_amdgcn_update_dpp((int)Q[c], (int)P[c], 0x128, 0xf, 0x3, false);
        }
    }
    // fragments j, j + 1 of row tile i in 16 bits: 16 bytes of lane group 0, 2 are columns
    // 0-7, 8-15 of the even fragment, of 1, 3 those of the odd one
    template <int i, int j>
    __device__ __forceinline__ u32x4 pair16() const {
        typedef typename ElemOf<C::DT>::type t2 __attribute__((ext_vector_type(2)));
        typedef typename ElemOf<C::DT>::type T;
        u32x4 v;
        static_for<0, 2, 1>([&](auto hc) {
            constexpr int h = decltype(hc)::value;
            const t2 even = {(T)get<i, j, 2 * h>(), (T)get<i, j, 2 * h + 1>()};
            const t2 odd = {(T)get<i, j + 1, 2 * h>(), (T)get<i, j + 1, 2 * h + 1>()};
            const auto r = __builtin_amdgcn_permlane16_swap(__builtin_bit_cast(uint32_t, even),
                                                            __builtin_bit_cast(uint32_t, odd), false, false);
            v[h] = r[0];
            v[2 + h] = r[1];
        });
        return v;
    }
    template <int i, int j>
    __device__ __forceinline__ u32x4 quad32() const {
        return __builtin_bit_cast(u32x4, f32x4{get<i, j, 0>(), get<i, j, 1>(), get<i, j, 2>(), get<i, j, 3>()});
    }
    // PAST: with the non-temporal hint (GroupedParams::past)
    template <bool PAST>
    __device__ __forceinline__ static void put(char *at, const u32x4 &v) {
        if constexpr (PAST) __builtin_nontemporal_store(v, reinterpret_cast<u32x4 *>(at));
        else *reinterpret_cast<u32x4 *>(at) = v;
    }
    // A store takes two fragments (fp32) or four (16 bits) of the wave's columns; a wave
    // with two of 16 bits stores 64 bytes of each of 16 rows.
    static constexpr bool short_rows(bool f32) { return !f32 && TN % 4 != 0; }
    // row: this lane's first, `first` in the tile (ORDERED: of row 0 of C); half: 8 rows.
    // MASKED: rows below `rows` and columns below `cols`, counted from this lane's first
    // (whole units of 16 bytes: the caller's condition)
    template <bool F32, bool PAST, bool MASKED>
    __device__ __forceinline__ void store_whole(char *row, int64_t half, int first, int rows, int cols) const {
        auto out = [&](char *at, const u32x4 &v, int r, int c) {
            if (!MASKED || (r < rows && c < cols)) put<PAST>(at, v);
        };
        static_assert(TN % 2 == 0, "whole 64 bytes of a wave's columns");
        char *const column = row;
        static_for<0, C::TM, 1>([&](auto ic) {
            constexpr int i = decltype(ic)::value;
            char *second = row + half;
            if constexpr (ORDERED) {
                auto place = [&](int r) {
                    if (MASKED && r >= rows) r = rows > 0 ? rows - 1 : -first;
                    return column + row_in(order, first + r, total) * (half / 8);
                };
                row = place(16 * i);
                if (!short_rows(F32)) second = place(16 * i + 8);
            }
            if constexpr (short_rows(F32)) {
                static_for<0, TN, 2>([&](auto jc) {
                    constexpr int j = decltype(jc)::value;
                    if constexpr (C::DT != DT_F32) out(row + 32 * j, pair16<i, j>(), 16 * i, 16 * j);
                });
            } else if constexpr (F32) {
                static_for<0, TN, 2>([&](auto jc) {
                    constexpr int j = decltype(jc)::value;
                    u32x4 low, high;
                    trade_rows(quad32<i, j>(), quad32<i, j + 1>(), low, high);
                    out(row + 64 * j, low, 16 * i, 16 * j);
                    out(second + 64 * j, high, 16 * i + 8, 16 * j);
                });
            } else if constexpr (C::DT != DT_F32) {
                static_for<0, TN, 4>([&](auto jc) {
                    constexpr int j = decltype(jc)::value;
                    u32x4 low, high;
                    trade_rows(pair16<i, j>(), pair16<i, j + 2>(), low, high);
                    out(row + 32 * j, low, 16 * i, 16 * j);
                    out(second + 32 * j, high, 16 * i + 8, 16 * j);
                });
            }
            if constexpr (!ORDERED) row += 2 * half;
        });
    }
    __device__ __forceinline__ void store(char *Cp, int64_t at, int64_t ldc, int m_left, int n_left, bool c_f32,
                                          bool past) const {
        const int g = lane / 16, m = (wave / C::WAVES_N) * C::WTM + lane % 16, n = (wave % C::WAVES_N) * WTN;
        const bool f32 = C::DT == DT_F32 || c_f32;
        const int size = f32 ? 4 : 2;
        char *first = Cp + at * size;
        const bool wide = ldc * size % 16 == 0 && reinterpret_cast<uintptr_t>(first) % 16 == 0;
        const int unit = 16 / size;
        if (wide && (n_left >= BN || n_left % unit == 0)) {
            const bool is_short = short_rows(f32);
            const int rm = (wave / C::WAVES_N) * C::WTM + (is_short ? lane % 16 : lane % 8);
            const int rn = n + (f32 ? 4 * g : 8 * (g / 2) + 16 * (g % 2)) + (is_short ? 0 : 64 / size * (lane % 16 / 8));
            char *row = first + ((ORDERED ? 0 : (int64_t)rm * ldc) + rn) * size;
            const int64_t half = 8 * ldc * size;
            if (m_left >= C::BM && n_left >= BN) {
                if (f32 && past) store_whole<true, true, false>(row, half, rm, 0, 0);
                else if (f32) store_whole<true, false, false>(row, half, rm, 0, 0);
                else if (past) store_whole<false, true, false>(row, half, rm, 0, 0);
                else store_whole<false, false, false>(row, half, rm, 0, 0);
            } else {
                if (f32) store_whole<true, false, true>(row, half, rm, m_left - rm, n_left - rn);
                else store_whole<false, false, true>(row, half, rm, m_left - rm, n_left - rn);
            }
            return;
        }
        const bool wide4 = ldc % 4 == 0 && reinterpret_cast<uintptr_t>(first) % 16 == 0;
        static_for<0, C::TM, 1>([&](auto ic) {
            constexpr int i = decltype(ic)::value;
            if (m + 16 * i < m_left) {
                int64_t place = m + 16 * i;
                if constexpr (ORDERED) place = row_in(order, m + 16 * i, total);
                const int64_t row = at + place * ldc + n + 4 * g;
                static_for<0, TN, 1>([&](auto jc) {
                    constexpr int j = decltype(jc)::value;
                    const f32x4 v = {get<i, j, 0>(), get<i, j, 1>(), get<i, j, 2>(), get<i, j, 3>()};
                    const int left = n_left - n - 4 * g - 16 * j;
                    if (left > 0) store4<C::DT>(Cp, row + 16 * j, left, c_f32, wide4, v);
                });
            }
        });
    }
};

template <class C, bool KS> using OperandA = RingOperand<typename std::conditional<KS, typename SwapCfg<C>::type, C>::type, KS, C::TM>;
template <class C, bool KS> using OperandB = RingOperand<typename std::conditional<KS, C, typename SwapCfg<C>::type>::type, KS, C::TN>;

template <class C, bool A_KS, bool B_KS, int STAGES, class OA_ = OperandA<C, A_KS>, class OB_ = OperandB<C, B_KS>>
struct GroupedTile {
    using OA = OA_;
    using OB = OB_;
    static constexpr int COPIES = OA::PER + OB::PER;
    static constexpr int LDS = STAGES * (OA::REGION + OB::REGION);
    static constexpr int READS = C::TM * OA::PIECES + C::TN * OB::PIECES;
    static constexpr int NMFMA = C::MFMA_PER_READ * C::TM * C::TN;
    // a read's distance from its base, the LDS copy included, is the 16-bit immediate of a DS instruction
    static_assert((STAGES - 1) * OA::REGION + OA::REACH < 65536 && (STAGES - 1) * OB::REGION + OB::REACH < 65536,
                  "DS offsets");

    OA a;
    OB b;
    AccTiles<C> acc;
    int K, nk, ndma;            // ndma: K tiles copied straight to LDS (all, or all but the last)
    int wave, lane;
    u32x4 tail[COPIES];

    // whole_chunks: no chunk of the last K tile that the copies bring passes a matrix's end
    __device__ __forceinline__ void begin(int K_, bool whole_chunks) {
        lane = threadIdx.x & 63;
        wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        K = K_;
        nk = (K + C::BK - 1) / C::BK;
        ndma = (K % C::BK == 0 && whole_chunks) || nk == 0 ? nk : nk - 1;
    }
    __device__ __forceinline__ void init(const char *A, int64_t lda, int m_left, const char *B, int64_t ldb, int n_left,
                                         int K_, char *smem) {
        begin(K_, (!A_KS || m_left >= C::BM || m_left % C::CHUNK == 0) &&
                      (!B_KS || n_left >= C::BN || n_left % C::CHUNK == 0));
        const uint32_t lds0 = lds_address(smem);
        b.init(B, ldb, n_left, (wave % C::WAVES_N) * C::WTN, lds0, lane, wave);
        a.init(A, lda, m_left, (wave / C::WAVES_N) * C::WTM, lds0 + STAGES * OB::REGION, lane, wave);
        acc.zero();
    }
    __device__ __forceinline__ void copy(int stage) {
        a.copy(stage);
        b.copy(stage);
    }
    __device__ __forceinline__ void tail_load() {
        const int64_t k0 = (int64_t)(nk - 1) * C::BK;
        a.tail_load(k0, K, &tail[0]);
        b.tail_load(k0, K, &tail[OA::PER]);
    }
    // at most `later` later tiles' copies in flight, or AHEAD if that is less
    template <int AHEAD>
    __device__ __forceinline__ static void wait_copies(int later) {
        static_assert(AHEAD * COPIES < 64, "the counter's range");
        if constexpr (AHEAD == 0) {
            wait_vmcnt<0>();
        } else {
            if (later >= AHEAD) wait_vmcnt<AHEAD * COPIES>();
            else wait_copies<AHEAD - 1>(later);
        }
    }
    // Wait until this wave's share of tile t is in LDS copy `stage`, at most AHEAD
    // later tiles being in flight; the last tile is stored from its registers.
    template <int AHEAD>
    __device__ __forceinline__ void land(int t, int stage) {
        if (t < ndma) {
            wait_copies<AHEAD>(ndma - 1 - t);
        } else {
            wait_vmcnt<0>();
            a.tail_store(stage, &tail[0]);
            b.tail_store(stage, &tail[OA::PER]);
        }
        wait_lds();
    }
    __device__ __forceinline__ void read_piece(int stage, int r, u32x4 (&fa)[C::TM], u32x4 (&fb)[C::TN]) const {
        constexpr int NA = C::TM * OA::PIECES;
        if (r < NA) a.read(stage, r / OA::PIECES, r % OA::PIECES, fa[r / OA::PIECES]);
        else b.read(stage, (r - NA) / OB::PIECES, (r - NA) % OB::PIECES, fb[(r - NA) / OB::PIECES]);
    }
    // MFMA q of a K tile (step e outermost: an accumulator's are TM x TN apart)
    template <bool FIRST, int q>
    __device__ __forceinline__ void mma(const u32x4 (&fa)[C::TM], const u32x4 (&fb)[C::TN]) {
        constexpr int e = q / (C::TM * C::TN), i = (q / C::TN) % C::TM, j = q % C::TN;
        acc.template mma<FIRST && e == 0>(i, j, fb[j], fa[i], e);
    }

    // All waves in step: wait for tile kt, one barrier, copy tile kt + STAGES - 1
    // into the copy just released, multiply tile kt.
    __device__ __forceinline__ void run_ring() {
        if (nk == 0) return;
        if (ndma < nk) tail_load();
#pragma unroll
        for (int t = 0; t < STAGES - 1; ++t)
            if (t < ndma) copy(t);
        int cur = 0, nxt = STAGES - 1;
        auto step = [&](int kt, auto first) {
            land<STAGES - 2>(kt, cur);
            block_barrier();
            if (kt + STAGES - 1 < ndma) copy(nxt);
            u32x4 fa[C::TM], fb[C::TN];
#pragma unroll
            for (int r = 0; r < READS; ++r) read_piece(cur, r, fa, fb);
            static_for<0, NMFMA, 1>([&](auto q) { mma<decltype(first)::value, decltype(q)::value>(fa, fb); });
            cur = cur + 1 == STAGES ? 0 : cur + 1;
            nxt = nxt + 1 == STAGES ? 0 : nxt + 1;
        };
        step(0, std::true_type{});
        for (int kt = 1; kt < nk; ++kt) step(kt, std::false_type{});
        acc.settle();
    }

    // The software pipeline of gemm_ring.hpp (one wave per SIMD, a K tile's
    // fragments in registers, twice): multiply tile t from (fa, fb) while tile
    // t + 1 is read into (na, nb) and tile t + STAGES copied into tile t's copy.
    // STEADY: both exist; else both are conditional.
    template <bool STEADY, bool FIRST = false>
    __device__ __forceinline__ void iter(int t, int cur, int next, u32x4 (&fa)[C::TM], u32x4 (&fb)[C::TN],
                                         u32x4 (&na)[C::TM], u32x4 (&nb)[C::TN]) {
        static_assert(READS <= NMFMA, "one fragment read per MFMA at most");
        const bool more = STEADY || t + 1 < nk;
        if (STEADY) wait_vmcnt<(STAGES - 2) * COPIES>();
        else if (more) land<STAGES - 2>(t + 1, next);
        wait_lds();
        __builtin_amdgcn_sched_barrier(0);
        block_barrier();
        __builtin_amdgcn_sched_barrier(0);
        if (STEADY) {
            static_for<0, NMFMA, 1>([&](auto qc) {
                constexpr int q = decltype(qc)::value;
                mma<FIRST, q>(fa, fb);
                if constexpr (q < READS) read_piece(next, q, na, nb);
                if constexpr (q == NMFMA / 4 - 1) a.copy(cur);
                if constexpr (q == 3 * NMFMA / 4 - 1) b.copy(cur);
                __builtin_amdgcn_sched_barrier(0);
            });
        } else {
            if (more) {
#pragma unroll
                for (int r = 0; r < READS; ++r) read_piece(next, r, na, nb);
            }
            if (t + STAGES < ndma) copy(cur);
            static_for<0, NMFMA, 1>([&](auto q) { mma<FIRST, decltype(q)::value>(fa, fb); });
        }
    }
    __device__ __forceinline__ void run_pipe() {
        static_assert(STAGES == 4, "four tiles per trip cycle the LDS copies");
        if (nk == 0) return;
        // a last tile that goes through registers: with at most STAGES copied tiles it is
        // landed by the prologue or the first iteration, and loaded before any copy
        const bool cut = ndma < nk, early = cut && ndma <= STAGES;
        if (early) tail_load();
#pragma unroll
        for (int t = 0; t < STAGES; ++t)
            if (t < ndma) copy(t);
        land<STAGES - 1>(0, 0);
        __builtin_amdgcn_sched_barrier(0);
        block_barrier();
        __builtin_amdgcn_sched_barrier(0);
        u32x4 a0[C::TM], b0[C::TN], a1[C::TM], b1[C::TN];
#pragma unroll
        for (int r = 0; r < READS; ++r) read_piece(0, r, a0, b0);
        if (STAGES < ndma) iter<true, true>(0, 0, 1, a0, b0, a1, b1);
        else iter<false, true>(0, 0, 1, a0, b0, a1, b1);
        int t = 1;
        for (; t + 3 + STAGES < ndma; t += 4) {
            iter<true>(t, 1, 2, a1, b1, a0, b0);
            iter<true>(t + 1, 2, 3, a0, b0, a1, b1);
            iter<true>(t + 2, 3, 0, a1, b1, a0, b0);
            iter<true>(t + 3, 0, 1, a0, b0, a1, b1);
        }
        int cur = t % STAGES;
        // the last tile's loads are younger than some copies, which only makes a wait longer
        if (cut && !early) tail_load();
        for (; t + 1 < nk; t += 2) {
            const int c1 = (cur + 1) % STAGES, c2 = (cur + 2) % STAGES;
            iter<false>(t, cur, c1, a1, b1, a0, b0);
            iter<false>(t + 1, c1, c2, a0, b0, a1, b1);
            cur = c2;
        }
        if (t < nk) iter<false>(t, cur, (cur + 1) % STAGES, a1, b1, a0, b0);
        acc.settle();
    }

    // C's tile: rows m < m_left, columns n < n_left, from its element `at`.
    __device__ __forceinline__ void store(char *Cp, int64_t at, int64_t ldc, int m_left, int n_left, bool c_f32,
                                          bool past) const {
        const auto value = [&](auto i, auto j, auto v) {
            return acc.get(decltype(i)::value, decltype(j)::value, decltype(v)::value);
        };
        TileStore<C, C::TN, decltype(value)>{value, lane, wave}.store(Cp, at, ldc, m_left, n_left, c_f32, past);
    }
};

// ---- which tile a workgroup takes ------------------------------------------------------
// Products over rows: only the device knows every group's (an expert's, or the
// rows' without one) rows.  The grid holds the most work there can be; each wave
// sums the groups' tile rows, 64 groups a step, and workgroups past the total
// end at once.
//
// A kernel of 256 x 256 tiles has pieces of 128 x 128 too, for what would leave
// the GPU half idle: a group's last tile row when it has at most 128 rows, and
// the tiles past the last whole round of 256 when there are at most kSplitRound,
// as four pieces each.
//
// Ids are dealt to the XCDs in contiguous runs, walked in groups of 8 tile rows.
constexpr uint32_t kRound = 256, kSplitRound = 128;

struct RowTile {
    bool piece;
    int g, lo, rows, m0, n0;      // rows: from m0 to the group's end
};

__device__ __forceinline__ int wave_inclusive(int v, int lane) {
    for (int d = 1; d < 64; d *= 2) {
        const int up = __shfl_up(v, d);
        if (lane >= d) v += up;
    }
    return v;
}

// id-th of n, so that the ids that one XCD receives (id % 8) are a contiguous run
__device__ __forceinline__ uint32_t xcd_run(uint32_t id, uint32_t n) {
    const uint32_t per = n / 8, rem = n % 8, x = id % 8;
    return x * per + (x < rem ? x : rem) + id / 8;
}

// tile id of rows x cols tiles, by columns within groups of 8 tile rows
__device__ __forceinline__ void grouped_order(uint32_t id, uint32_t rows, uint32_t cols, int &tm, int &tn) {
    const uint32_t group = id / (8 * cols), first = group * 8;
    const uint32_t here = rows - first < 8 ? rows - first : 8;
    const uint32_t in = id - first * cols;
    tm = (int)(first + in % here);
    tn = (int)(in / here);
}

// BM: 256 with pieces of 128 (PIECES), or a tile of BM x BN alone.
template <int BM, int BN, bool PIECES>
__device__ __forceinline__ bool row_tile(const GroupedParams &p, RowTile &t) {
    const int lane = threadIdx.x & 63;
    const int groups = p.experts + 1;
    const uint32_t tiles_n = (p.N + BN - 1) / BN;
    RowSpan s = {0, 0};
    int big = 0, small = 0, big_incl = 0, small_incl = 0;
    auto look = [&](int base) {
        s = base + lane < groups ? rows_of(p.offsets, base + lane, p.experts, p.rows) : RowSpan{0, 0};
        const int n = s.hi - s.lo, rest = n % BM;
        if (PIECES) {
            big = n / BM + (rest > BM / 2);
            small = rest > 0 && rest <= BM / 2;
            small_incl = wave_inclusive(small, lane);
        } else {
            big = (n + BM - 1) / BM;
        }
        big_incl = wave_inclusive(big, lane);
    };
    uint32_t total_b = 0, total_s = 0;
    for (int base = 0; base < groups; base += 64) {
        look(base);
        total_b += __builtin_amdgcn_readlane(big_incl, 63);
        if (PIECES) total_s += __builtin_amdgcn_readlane(small_incl, 63);
    }
    const uint32_t tiles = total_b * tiles_n, left = PIECES ? tiles % kRound : 0;
    const uint32_t whole = PIECES && left <= kSplitRound ? tiles - left : tiles;   // tiles taken as they are
    uint32_t id = blockIdx.x;
    int row;              // which tile row, among the big ones or the small ones
    int half_m = 0;       // a piece's place in a split tile's rows
    bool of_small = false;
    t.piece = false;
    if (id < whole) {
        int tn;
        grouped_order(xcd_run(id, whole), total_b, tiles_n, row, tn);
        t.n0 = tn * BN;
    } else {
        if (!PIECES) return false;
        id -= whole;
        t.piece = true;
        int tn;
        if (id < 4 * (tiles - whole)) {
            grouped_order(whole + id / 4, total_b, tiles_n, row, tn);
            half_m = id / 2 % 2;
            t.n0 = tn * BN + (int)(id % 2) * (BN / 2);
        } else {
            id -= 4 * (tiles - whole);
            const uint32_t pieces_n = (p.N + BN / 2 - 1) / (BN / 2);
            if (id >= total_s * pieces_n) return false;
            of_small = true;
            row = (int)(id / pieces_n);
            t.n0 = (int)(id % pieces_n) * (BN / 2);
        }
        if (t.n0 >= p.N) return false;
    }
    int before = 0;
    for (int base = 0; base < groups; base += 64) {
        if (groups > 64) look(base);
        const int incl = of_small ? small_incl : big_incl, mine = of_small ? small : big;
        const int here = __builtin_amdgcn_readlane(incl, 63);
        if (row < before + here) {
            const int l = __builtin_ctzll(__ballot(before + incl > row));
            const int first = before + __builtin_amdgcn_readlane(incl - mine, l);
            t.g = base + l;
            t.lo = __builtin_amdgcn_readlane(s.lo, l);
            const int n = __builtin_amdgcn_readlane(s.hi, l) - t.lo;
            t.m0 = of_small ? n / BM * BM : (row - first) * BM + half_m * (BM / 2);
            t.rows = n - t.m0;
            return t.rows > 0;
        }
        before += here;
    }
    return false;
}

template <class C, bool A_KS, bool B_KS, bool PIPE, int STAGES>
__device__ __forceinline__ void run_tile_of(const GroupedParams &p, char *smem, const char *A, int64_t lda, int m_left,
                                            const char *B, int n_left, int K, int64_t c_at) {
    GroupedTile<C, A_KS, B_KS, STAGES> tile;
    tile.init(A, lda, m_left, B, p.ldb, n_left, K, smem);
    if constexpr (PIPE) tile.run_pipe();
    else tile.run_ring();
    tile.store(p.C, c_at, p.ldc, m_left, n_left, p.c_f32, p.past);
}

// P: the configuration of the pieces (C itself: none).
template <class C, class P, bool B_KS, bool PIPE, int STAGES>
__global__ __launch_bounds__(C::THREADS, C::OCCUPANCY) void grouped_tile_kernel(GroupedParams p) {
    constexpr bool PIECES = !std::is_same<C, P>::value;
    static_assert(!PIECES || (P::BM * 2 == C::BM && P::BN * 2 == C::BN && P::THREADS == C::THREADS), "quarters");
    __shared__ __attribute__((aligned(1024))) char smem[GroupedTile<C, false, B_KS, STAGES>::LDS];
    RowTile t;
    if (!row_tile<C::BM, C::BN, PIECES>(p, t)) return;
    const bool dead = t.g == p.experts;
    const int64_t row = t.lo + t.m0;
    const char *A = p.A + row * p.lda * C::ELEM;
    const char *B = p.B + ((dead ? 0 : (int64_t)t.g * p.sB) + (B_KS ? (int64_t)t.n0 : t.n0 * p.ldb)) * C::ELEM;
    const int K = dead ? 0 : p.K;
    if (PIECES && t.piece)
        run_tile_of<P, false, B_KS, PIPE, STAGES>(p, smem, A, p.lda, t.rows, B, p.N - t.n0, K, row * p.ldc + t.n0);
    else
        run_tile_of<C, false, B_KS, PIPE, STAGES>(p, smem, A, p.lda, t.rows, B, p.N - t.n0, K, row * p.ldc + t.n0);
}

// The gradient with respect to B: experts x tiles_m x tiles_n tiles, whose work
// goes with their expert's rows.  Every expert's tiles are dealt to all eight XCDs,
// a contiguous run each (an XCD of its own for a popular expert would work on
// alone); workgroups go to them in turn, so that no gap may lie between experts (a
// multiple of eight for each left XCDs idle: 256 experts of 128 x 128 bf16, 65536 rows, 41
// us and 10 without, 10 of 1280 x 1280 67.5 and 41.5).  Up to 64 experts go in order of
// their rows, the most first, so that the last tiles to end are short ones (8 uneven
// experts of 2048 x 4096: 220 -> 214 us; the order costs a small tile more than it gives:
// 33 of 257 x 1000 19.0 -> 20.5, so only the large ones).
template <class C, bool PIPE, int STAGES>
__global__ __launch_bounds__(C::THREADS, C::OCCUPANCY) void wgrad_tile_kernel(GroupedParams p) {
    __shared__ __attribute__((aligned(1024))) char smem[GroupedTile<C, true, true, STAGES>::LDS];
    const uint32_t tiles_m = (p.M + C::BM - 1) / C::BM, tiles_n = (p.N + C::BN - 1) / C::BN, tiles = tiles_m * tiles_n;
    int g = (int)(blockIdx.x / tiles);
    const uint32_t id = xcd_run(blockIdx.x % tiles, tiles);
    int tm, tn;
    grouped_order(id, tiles_m, tiles_n, tm, tn);
    const int m0 = tm * C::BM, n0 = tn * C::BN;
    if (PIPE && p.experts > 1 && p.experts <= 64) {
        const int lane = threadIdx.x & 63;
        const RowSpan of = lane < p.experts ? rows_of(p.offsets, lane, p.experts, p.rows) : RowSpan{0, -1};
        const int mine = of.hi - of.lo;
        int rank = 0;
        for (int e = 0; e < p.experts; ++e) {
            const int n = __builtin_amdgcn_readlane(mine, e);
            rank += n > mine || (n == mine && e < lane);
        }
        g = __builtin_ctzll(__ballot(rank == g));
    }
    const RowSpan s = rows_of(p.offsets, g, p.experts, p.rows);
    const int lo = __builtin_amdgcn_readfirstlane(s.lo), K = __builtin_amdgcn_readfirstlane(s.hi) - lo;
    run_tile_of<C, true, true, PIPE, STAGES>(p, smem, p.A + ((int64_t)lo * p.lda + m0) * C::ELEM, p.lda, p.M - m0,
                                     p.B + ((int64_t)lo * p.ldb + n0) * C::ELEM, p.N - n0, K,
                                     (int64_t)g * p.sC + (int64_t)m0 * p.ldc + n0);
}

}  // namespace tg
