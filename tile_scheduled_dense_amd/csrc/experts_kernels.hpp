// experts_kernels.hpp -- instantiations and launches of the expert products'
// kernels (experts.hpp) by their plans (experts_plan.hpp), included by one
// translation unit per input type.
#pragma once

#include <hip/hip_runtime.h>

#include "experts_plan.hpp"

namespace tg {
namespace {

inline tg_status launched() { return hipGetLastError() == hipSuccess ? TG_OK : TG_ERR_LAUNCH; }

template <int DT, bool TRANS>
tg_status launch_stream(const GroupedParams &p, const ProductPlan &plan, hipStream_t s) {
    const int waves = plan.info.waves;
    const unsigned lds = waves * StreamShape<DT, TRANS>::FRAGS * 1024;
    hipLaunchKernelGGL((grouped_stream_kernel<DT, TRANS>), dim3((unsigned)plan.gx, plan.gy, plan.gz), dim3(64 * waves), lds,
                       s, p);
    return launched();
}

template <int DT, int GROUP, int NT>
tg_status launch_q4_as(const Q4Params &p, const ProductPlan &plan, hipStream_t s) {
    const int waves = plan.info.waves;
    const unsigned lds = waves * Q4Rows<DT>::LDS * 16;
    hipLaunchKernelGGL((q4_kernel<DT, GROUP, NT>), dim3((unsigned)plan.gx, plan.gy, plan.gz), dim3(64 * waves), lds, s, p);
    return launched();
}

template <int DT, int GROUP>
tg_status launch_q4_group(const Q4Params &p, hipStream_t s) {
    const ProductPlan plan = plan_q4<DT>(p.experts, p.rows, p.N, p.K);
    if constexpr (DT != DT_F32) {
        if (plan.info.tile_n == 32) return launch_q4_as<DT, GROUP, 2>(p, plan, s);
    }
    return launch_q4_as<DT, GROUP, 1>(p, plan, s);
}

template <int DT> using Tile256 = RingCfg<DT, 256, 256, 2, 2, 16>;
template <int DT> using Tile128 = RingCfg<DT, 128, 128, 2, 2, 16>;
using Tile64F32 = RingCfg<DT_F32, 64, 64, 2, 2, 16>;

// P: the pieces' configuration (C itself: none).
template <class C, class P, bool B_KS, bool PIPE, int STAGES>
tg_status launch_tiles(const GroupedParams &p, const ProductPlan &plan, hipStream_t s) {
    if (!plan.fits()) return TG_ERR_UNSUPPORTED;
    hipLaunchKernelGGL((grouped_tile_kernel<C, P, B_KS, PIPE, STAGES>), dim3((unsigned)plan.gx), dim3(C::THREADS), 0, s, p);
    return launched();
}

template <class C, bool PIPE, int STAGES>
tg_status launch_wgrad_tiles(const GroupedParams &p, const ProductPlan &plan, hipStream_t s) {
    if (!plan.fits()) return TG_ERR_UNSUPPORTED;
    hipLaunchKernelGGL((wgrad_tile_kernel<C, PIPE, STAGES>), dim3((unsigned)plan.gx), dim3(C::THREADS), 0, s, p);
    return launched();
}

template <int DT, bool TRANS>
tg_status launch_grouped_as(const GroupedParams &p, hipStream_t s) {
    const ProductPlan plan = plan_grouped_as<DT, TRANS>(p.experts, p.rows, p.N, p.K);
    if (plan.info.kernel == TG_EXPERTS_STREAM) return launch_stream<DT, TRANS>(p, plan, s);
    if (plan.info.tile_m == 256) return launch_tiles<Tile256<DT>, Tile128<DT>, !TRANS, true, 4>(p, plan, s);
    if constexpr (DT == DT_F32) return launch_tiles<Tile64F32, Tile64F32, !TRANS, true, 4>(p, plan, s);
    else return launch_tiles<Tile128<DT>, Tile128<DT>, !TRANS, false, 3>(p, plan, s);
}

}  // namespace

template <int DT>
tg_status launch_grouped(const GroupedParams &p, bool transposed, hipStream_t s) {
    return transposed ? launch_grouped_as<DT, true>(p, s) : launch_grouped_as<DT, false>(p, s);
}

template <int DT>
tg_status launch_wgrad(const GroupedParams &p, hipStream_t s) {
    const ProductPlan plan = plan_wgrad<DT>(p.experts, p.rows, p.M, p.N);
    if (plan.info.kernel == TG_EXPERTS_NARROW) {
        const int width = p.M < p.N ? plan.info.tile_n : plan.info.tile_m;
        hipLaunchKernelGGL((wgrad_narrow_kernel<DT>), dim3((unsigned)plan.gx, plan.gy), dim3(1024), 0, s, p, width);
        return launched();
    }
    if (plan.info.tile_m == 256) return launch_wgrad_tiles<Tile256<DT>, true, 4>(p, plan, s);
    if constexpr (DT == DT_F32) return launch_wgrad_tiles<Tile64F32, true, 4>(p, plan, s);
    else if (plan.info.pipeline) return launch_wgrad_tiles<Tile128<DT>, true, 4>(p, plan, s);
    else return launch_wgrad_tiles<Tile128<DT>, false, 3>(p, plan, s);
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
