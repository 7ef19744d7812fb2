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
template <int DT> using Tile64 = RingCfg<DT, 64, 64, 2, 2, 16>;

// Tiles: whole ones and pieces, or with K split and a second launch that adds up.
template <class C, class P, bool KS, bool ORDERED, bool PIPE, int STAGES>
tg_status launch_adapter_tiles(const AdapterParams &p, const ProductPlan &plan, hipStream_t s) {
    const dim3 grid((unsigned)plan.gx), block(C::THREADS);
    if (p.splits > 1) {
        hipLaunchKernelGGL((adapters_tile_split_kernel<C, KS, ORDERED, PIPE, STAGES>), grid, block, 0, s, p);
        const tg_status st = launched();
        if (st != TG_OK) return st;
        const int64_t sums = cdiv((int64_t)p.rows * cdiv(p.N, 4), 256);
        hipLaunchKernelGGL((adapters_sum_kernel<C::DT>), dim3((unsigned)sums), dim3(256), 0, s, p);
        return launched();
    }
    hipLaunchKernelGGL((adapters_tile_kernel<C, P, KS, ORDERED, PIPE, STAGES>), grid, block, 0, s, p);
    return launched();
}

template <int DT, bool KS, bool ORDERED>
tg_status launch_adapters_many(const AdapterParams &p, const AdapterPlan &plan, hipStream_t s) {
    if (p.rank > 0) {
        const dim3 grid((unsigned)plan.low.gx, plan.low.gy, plan.low.gz);
        hipLaunchKernelGGL((shrink_tile_kernel<Tile64<DT>, KS, ORDERED, 4>), grid, dim3(256), 0, s, p);
        tg_status st = launched();
        if (st != TG_OK) return st;
        const int64_t quads = cdiv((int64_t)p.rows * (p.ld_low / 4), 256);
        if (!grid_fits(quads, 256)) return TG_ERR_UNSUPPORTED;
        hipLaunchKernelGGL((shrink_join_kernel<DT>), dim3((unsigned)quads), dim3(256), 0, s, p);
        st = launched();
        if (st != TG_OK) return st;
    }
    if constexpr (DT == DT_F32) {
        return launch_adapter_tiles<Tile64<DT>, Tile64<DT>, KS, ORDERED, true, 4>(p, plan.product, s);
    } else {
        if (plan.product.info.tile_m == 256)
            return launch_adapter_tiles<Tile256<DT>, Tile128<DT>, KS, ORDERED, true, 4>(p, plan.product, s);
        return launch_adapter_tiles<Tile128<DT>, Tile128<DT>, KS, ORDERED, false, 3>(p, plan.product, s);
    }
}

template <int DT, bool TRANS>
tg_status launch_adapters_as(AdapterParams p, void *workspace, hipStream_t s) {
    using S = StreamShape<DT, TRANS>;
    const AdapterPlan plan = plan_adapters_as<DT, TRANS>(p.experts, p.rows, p.N, p.K, p.rank);
    if (!plan.product.fits() || !plan.low.fits() ||
        !grid_fits(plan.product.gx + plan.low.gx, 64 * plan.product.info.waves))
        return TG_ERR_UNSUPPORTED;
    p.splits = plan.splits;
    p.t_splits = plan.t_splits;
    p.part = static_cast<float *>(workspace);
    p.part_t = reinterpret_cast<float *>(static_cast<char *>(workspace) + plan.part_bytes);
    p.low = static_cast<char *>(workspace) + plan.part_bytes + plan.part_t_bytes;
    p.ld_low = plan.ld_low;
    if (plan.form == ADAPTERS_TILES)
        return p.order ? launch_adapters_many<DT, !TRANS, true>(p, plan, s) : launch_adapters_many<DT, !TRANS, false>(p, plan, s);
    const int64_t low = p.rank > 0 ? plan.low.gx * plan.low.gy * plan.low.gz : 0, strips_t = cdiv(p.rank, S::COLS);
    const int64_t join = join_parts<TRANS>(p.N) * p.rows;
    if (!grid_fits(join, 256)) return TG_ERR_UNSUPPORTED;
    const dim3 grid((unsigned)(low + plan.product.gx)), block(64 * plan.product.info.waves);
    if (plan.form == ADAPTERS_STREAM)
        hipLaunchKernelGGL((adapters_few_kernel<DT, TRANS>), grid, block,
                           (unsigned)(plan.product.info.waves * S::FRAGS * 1024), s, p, (int)low, (int)cdiv(p.rows, 16),
                           (int)strips_t);
    else
        hipLaunchKernelGGL((adapters_split_kernel<Tile64<DT>, !TRANS, 4>), grid, block, 0, s, p, (int)low, (int)strips_t);
    const tg_status st = launched();
    if (st != TG_OK) return st;
    hipLaunchKernelGGL((adapters_join_kernel<DT, TRANS>), dim3((unsigned)join), dim3(256), 0, s, p);
    return launched();
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
    const int64_t join = cdiv((int64_t)(p.M[0] > p.M[1] ? p.M[0] : p.M[1]) * p.rank, 256);
    if (!grid_fits(plan.workgroups, 256) || !grid_fits(join, 256)) return TG_ERR_UNSUPPORTED;
    if (plan.workgroups > 0) {
        const dim3 grid((unsigned)plan.workgroups);
        if (p.rank <= 16) hipLaunchKernelGGL((adapters_wgrad_kernel<DT, 1>), grid, dim3(256), 0, s, p);
        else if (p.rank <= 32) hipLaunchKernelGGL((adapters_wgrad_kernel<DT, 2>), grid, dim3(256), 0, s, p);
        else hipLaunchKernelGGL((adapters_wgrad_kernel<DT, kWgradRank / 16>), grid, dim3(256), 0, s, p);
        const tg_status st = launched();
        if (st != TG_OK) return st;
    }
    if (join > 0)
        hipLaunchKernelGGL((adapters_wgrad_join_kernel<DT>), dim3((unsigned)join, (unsigned)p.adapters, 2), dim3(256), 0, s, p);
    return launched();
}

}  // namespace tg
