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
