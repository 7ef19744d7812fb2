// gate.hpp -- the elementwise part of a gated pair of projections and of its
// gradient, in fp32:
//
//   h = act(u) * v,   d_u = d_h * v * act'(u),   d_v = d_h * act(u)
//
// act by number: 0 the value itself, 1 ReLU, 2 GELU (x Phi(x)), 3 SiLU (x s(x), s the
// logistic function).  A NaN in u or v reaches h.
#pragma once

#include <hip/hip_runtime.h>

#include "gemm_kernel.hpp"

namespace tg {

enum { GATE_NONE = 0, GATE_RELU = 1, GATE_GELU = 2, GATE_SILU = 3, GATE_COUNT = 4 };

constexpr float kLog2e = 1.4426950408889634f;

// 1 / (1 + e^-x): e^-x overflows to infinity, whose reciprocal is 0
__device__ __forceinline__ float logistic(float x) {
    return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-x * kLog2e));
}

template <int ACT>
__device__ __forceinline__ float gate_act(float u) {
    if constexpr (ACT == GATE_RELU) return u < 0.0f ? 0.0f : u;
    else if constexpr (ACT == GATE_GELU) return gelu(u);
    else if constexpr (ACT == GATE_SILU) return u * logistic(u);
    else return u;
}

// act(u) and act'(u)
template <int ACT>
__device__ __forceinline__ void gate_both(float u, float &f, float &d) {
    if constexpr (ACT == GATE_RELU) {
        f = u < 0.0f ? 0.0f : u;
        d = u > 0.0f ? 1.0f : (u <= 0.0f ? 0.0f : u);      // a NaN stays one
    } else if constexpr (ACT == GATE_GELU) {
        // gelu'(x) = Phi(x) + x phi(x)
        const float phi = 0.3989422804014327f * __builtin_amdgcn_exp2f(-0.5f * kLog2e * u * u);
        const float cdf = normal_cdf(u);
        f = u * cdf;
        d = __builtin_fmaf(u, phi, cdf);
    } else if constexpr (ACT == GATE_SILU) {
        const float s = logistic(u);
        f = u * s;
        d = s * __builtin_fmaf(u, 1.0f - s, 1.0f);
    } else {
        f = u;
        d = 1.0f;
    }
}

// f with the activation's number as a constant
template <class F>
__device__ __forceinline__ void with_act(int act, const F &f) {
    if (act == GATE_SILU) f(std::integral_constant<int, GATE_SILU>{});
    else if (act == GATE_GELU) f(std::integral_constant<int, GATE_GELU>{});
    else if (act == GATE_RELU) f(std::integral_constant<int, GATE_RELU>{});
    else f(std::integral_constant<int, GATE_NONE>{});
}

}  // namespace tg
