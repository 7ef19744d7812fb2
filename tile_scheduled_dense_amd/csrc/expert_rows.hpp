// expert_rows.hpp -- what the kernels of the expert products share: element
// types, an expert's rows, the store of four neighbours of a result.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gemm_kernel.hpp"

namespace tg {

template <int DT> struct ElemOf;
template <> struct ElemOf<DT_F32> { typedef float type; };
template <> struct ElemOf<DT_BF16> { typedef __bf16 type; };
template <> struct ElemOf<DT_F16> { typedef _Float16 type; };

// Rows of expert g, clamped to what there is; g == experts: the rows without
// an expert.  offsets NULL: one expert with every row.
struct RowSpan {
    int lo, hi;
};
__device__ __forceinline__ RowSpan rows_of(const int32_t *offsets, int g, int experts, int rows) {
    if (!offsets) return g == 0 ? RowSpan{0, rows} : RowSpan{rows, rows};
    const int a = offsets[g];
    const int lo = a < 0 ? 0 : (a > rows ? rows : a);
    if (g == experts) return {lo, rows};
    const int b = offsets[g + 1];
    return {lo, b < lo ? lo : (b > rows ? rows : b)};
}

// Which expert has how many rows is known on the device alone, and all of them may have
// gone to one.  Products that take an expert's rows BM at a time have a workgroup for each
// group's (expert's, or the rows' without one) first tile, slots below 0, and behind those
// one for each of (rows - 1) / BM slots, which hold all further tiles: group g's start at
// offsets[g] / BM, which leaves it at least as many as it has further tiles.  A slot can only
// be of the last group that starts at or before it, which the lanes of a wave look for 64
// groups (or 64 runs of them) at a time.  (64 experts of 768 x 1024 f16, 512 rows: 25 us
// when all have 8, 8.4 when one has all; the first tile's workgroup taking them all in turn,
// 25 and 169.  2048 experts of 128 x 128 bf16, 8192 rows: 15 and 6.6, 15 and 1240.)
constexpr int kGridY = 32768;           // workgroups past it along y lie along z
__device__ __forceinline__ int slot_of(int experts) {
    return (int)(blockIdx.z * kGridY + blockIdx.y) - (experts + 1);
}
inline int64_t tiles_and_slots(int64_t rows, int64_t experts, int64_t bm) { return experts + 1 + (rows - 1) / bm; }

// The tile of `slot`, the same in the whole wave; false: none.  A wrong table finds wrong
// tiles inside the rows.
template <int BM>
__device__ __forceinline__ bool row_slot(const int32_t *offsets, int experts, int rows, int slot, int &g, RowSpan &tile) {
    int lo, hi, first;
    if (slot < 0) {
        g = slot + experts + 1;
        const RowSpan s = rows_of(offsets, g, experts, rows);
        lo = first = s.lo;
        hi = s.hi;
    } else if (!offsets) {
        g = 0;
        lo = 0;
        hi = rows;
        first = (slot + 1) * BM;
    } else {
        const int lane = threadIdx.x & 63, groups = experts + 1;
        auto at = [&](int i) {
            const int o = offsets[i < experts ? i : experts];
            return o < 0 ? 0 : (o > rows ? rows : o);
        };
        const int run = (groups + 63) / 64;      // 33 at most: a run's last neighbour is in a lane too
        int base = 0;
        if (run > 1) {
            const int i = lane * run;
            const uint64_t m = __ballot(i < groups && at(i) / BM <= slot);
            if (!m) return false;
            base = (63 - __builtin_clzll(m)) * run;
        }
        const int i = base + lane, o = at(i);
        const uint64_t m = __ballot(i < groups && (run == 1 || lane < run) && o / BM <= slot);
        if (!m) return false;
        const int l = 63 - __builtin_clzll(m);
        g = base + l;
        lo = __builtin_amdgcn_readlane(o, l);
        hi = g == experts ? rows : __builtin_amdgcn_readlane(o, l + 1);
        first = lo + (slot - lo / BM + 1) * BM;
    }
    tile = {first, hi - first < BM ? hi : first + BM};
    return first < hi;
}

// Write v = C[row][n .. n + 3] (n a multiple of 4), one rounding for a 16-bit C.
// wide: C's rows take 4 values in one aligned store.
template <int DT>
__device__ __forceinline__ void store4(char *C, int64_t at, int left, bool c_f32, bool wide, const f32x4 &v) {
    typedef typename ElemOf<DT>::type T;
    typedef T t4 __attribute__((ext_vector_type(4)));
    if (DT == DT_F32 || c_f32) {
        float *p = reinterpret_cast<float *>(C) + at;
        if (wide && left >= 4) {
            *reinterpret_cast<f32x4 *>(p) = v;
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (e < left) p[e] = v[e];
        }
    } else {
        T *p = reinterpret_cast<T *>(C) + at;
        const t4 x = {(T)v[0], (T)v[1], (T)v[2], (T)v[3]};
        if (wide && left >= 4) {
            *reinterpret_cast<t4 *>(p) = x;
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (e < left) p[e] = x[e];
        }
    }
}

}  // namespace tg
