// adapters_kernels.hpp -- instantiations and launches of the adapters' kernels (ffn.hpp),
// included by one translation unit per input type.
#pragma once

#include <hip/hip_runtime.h>

#include "ffn.hpp"
#include "ffn_plan.hpp"

namespace tg {
namespace {

inline tg_status launched() { return hipGetLastError() == hipSuccess ? TG_OK : TG_ERR_LAUNCH; }

template <int DT> using Tile256 = RingCfg<DT, 256, 256, 2, 2, 16>;
template <int DT> using Tile128 = RingCfg<DT, 128, 128, 2, 2, 16>;
using Tile64F32 = RingCfg<DT_F32, 64, 64, 2, 2, 16>;

template <class C, class P, bool B_KS, bool PIPE, int STAGES>
tg_status launch_adapter_tiles(const AdapterParams &p, const ProductPlan &plan, hipStream_t s) {
    const dim3 grid((unsigned)plan.gx), block(C::THREADS);
    if (p.order) hipLaunchKernelGGL((adapters_tile_kernel<C, P, B_KS, true, PIPE, STAGES>), grid, block, 0, s, p);
    else hipLaunchKernelGGL((adapters_tile_kernel<C, P, B_KS, false, PIPE, STAGES>), grid, block, 0, s, p);
    return launched();
}

template <int DT, bool TRANS>
tg_status launch_adapters_as(AdapterParams p, void *workspace, hipStream_t s) {
    using S = StreamShape<DT, TRANS>;
    const AdapterPlan plan = plan_adapters<DT, TRANS>(p.experts, p.rows, p.N, p.K, p.rank);
    const ProductPlan &product = plan.product;
    if (!product.fits()) return TG_ERR_UNSUPPORTED;
    const int64_t strips_t = cdiv(p.rank, S::COLS);
    p.splits = plan.splits;
    p.t_splits = plan.t_splits;
    if (plan.few) {
        p.part = static_cast<float *>(workspace);
        p.part_t = reinterpret_cast<float *>(static_cast<char *>(workspace) + plan.part_bytes);
        const int64_t row_tiles = cdiv(p.rows, 16), base = cdiv(p.N, S::COLS) * row_tiles * plan.splits;
        const int64_t join = cdiv(p.N, 1024) * p.rows;
        if (!grid_fits(join, 256)) return TG_ERR_UNSUPPORTED;
        hipLaunchKernelGGL((adapters_few_kernel<DT, TRANS>), dim3((unsigned)product.gx), dim3(64 * plan.waves),
                           plan.waves * S::FRAGS * 1024, s, p, (int)base, (int)row_tiles, (int)strips_t);
        const tg_status st = launched();
        if (st != TG_OK) return st;
        hipLaunchKernelGGL((adapters_join_kernel<DT, TRANS>), dim3((unsigned)join), dim3(256), 0, s, p);
        return launched();
    }
    p.low = static_cast<char *>(workspace);
    p.ld_low = plan.ld_low;
    if (p.rank > 0) {
        const ProductPlan low = plan_of(TG_EXPERTS_STREAM, 16, S::COLS, plan.t_waves, strips_t,
                                        tiles_and_slots(p.rows, p.experts, 16));
        hipLaunchKernelGGL((shrink_kernel<DT, TRANS>), dim3((unsigned)low.gx, low.gy, low.gz), dim3(64 * plan.t_waves),
                           plan.t_waves * S::FRAGS * 1024, s, p);
        const tg_status st = launched();
        if (st != TG_OK) return st;
    }
    if constexpr (DT == DT_F32) {
        return launch_adapter_tiles<Tile64F32, Tile64F32, !TRANS, true, 4>(p, product, s);
    } else {
        if (product.info.tile_m == 256)
            return launch_adapter_tiles<Tile256<DT>, Tile128<DT>, !TRANS, true, 4>(p, product, s);
        return launch_adapter_tiles<Tile128<DT>, Tile128<DT>, !TRANS, false, 3>(p, product, s);
    }
}

}  // namespace

template <int DT>
tg_status launch_adapters(const AdapterParams &p, bool transposed, void *workspace, hipStream_t s) {
    return transposed ? launch_adapters_as<DT, true>(p, workspace, s) : launch_adapters_as<DT, false>(p, workspace, s);
}

template <int DT>
tg_status launch_adapters_wgrad(const AdapterGradParams &q, void *workspace, hipStream_t s) {
    AdapterGradParams p = q;
    const AdapterGradPlan plan = plan_adapters_wgrad(p.adapters, p.rows, p.M[1], p.M[0], p.rank, DT == DT_F32);
    p.part[0] = static_cast<float *>(workspace);
    p.part[1] = reinterpret_cast<float *>(static_cast<char *>(workspace) + plan.part_bytes[0]);
    p.strips[0] = (int)plan.strips[0];
    p.strips[1] = (int)plan.strips[1];
    p.slots = (int)plan.slots;
    p.rank_tiles = (int)plan.rank_tiles;
    const int64_t longest = (int64_t)(p.M[0] > p.M[1] ? p.M[0] : p.M[1]) * p.rank, join = cdiv(longest, 256);
    if (!grid_fits(plan.workgroups, 256) || !grid_fits(join, 256)) return TG_ERR_UNSUPPORTED;
    if (plan.workgroups > 0) {
        hipLaunchKernelGGL((adapters_wgrad_kernel<DT>), dim3((unsigned)plan.workgroups), dim3(256), 0, s, p);
        const tg_status st = launched();
        if (st != TG_OK) return st;
    }
    if (join > 0)
        hipLaunchKernelGGL((adapters_wgrad_join_kernel<DT>), dim3((unsigned)join, (unsigned)p.adapters, 2), dim3(256), 0, s, p);
    return launched();
}

}  // namespace tg
