// gated_kernels.hpp -- instantiations and launches of the gated pair's kernels and its
// gate's gradient (ffn.hpp), included by one translation unit per input type.
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
template <int DT> using Tile64x128 = RingCfg<DT, 64, 128, 2, 2, 16>;

template <class C, class P, bool B_KS, bool PIPE, int STAGES>
tg_status launch_gated_tiles(const GatedParams &p, const ProductPlan &plan, hipStream_t s) {
    hipLaunchKernelGGL((gated_tile_kernel<C, P, B_KS, PIPE, STAGES>), dim3((unsigned)plan.gx), dim3(C::THREADS), 0, s, p);
    return launched();
}

template <int DT, bool TRANS>
tg_status launch_gated_as(const GatedParams &p, void *workspace, hipStream_t s) {
    const GatedPlan plan = plan_gated_as<DT, TRANS>(p.experts, p.rows, p.N, p.K);
    const ProductPlan &product = plan.product;
    if (!product.fits()) return TG_ERR_UNSUPPORTED;
    if (plan.splits > 0) {
        GatedParams f = p;
        f.part = static_cast<float *>(workspace);
        f.splits = workspace ? plan.splits : 1;
        const dim3 grid((unsigned)(product.gx / plan.splits * f.splits), product.gy, product.gz);
        if (product.info.kernel == TG_EXPERTS_STREAM)
            hipLaunchKernelGGL((gated_few_kernel<DT, TRANS>), grid, dim3(64 * product.info.waves),
                               (unsigned)(product.info.waves * StreamShape<DT, TRANS>::FRAGS * 1024), s, f);
        else
            hipLaunchKernelGGL((gated_split_kernel<Tile64x128<DT>, !TRANS, 4>), grid, dim3(256), 0, s, f);
        const tg_status st = launched();
        if (st != TG_OK || f.splits == 1) return st;
        const int64_t quads = (int64_t)p.rows * cdiv(p.N, 4);
        hipLaunchKernelGGL((gated_join_kernel<DT>), dim3((unsigned)cdiv(quads, 256)), dim3(256), 0, s, f);
        return launched();
    }
    if constexpr (DT == DT_F32) {
        return launch_gated_tiles<Tile64x128<DT>, Tile64x128<DT>, !TRANS, true, 4>(p, product, s);
    } else {
        if (product.info.tile_m == 256)
            return launch_gated_tiles<Tile256<DT>, Tile128<DT>, !TRANS, true, 4>(p, product, s);
        return launch_gated_tiles<Tile128<DT>, Tile128<DT>, !TRANS, false, 3>(p, product, s);
    }
}

template <class C, class P, bool B_KS, bool PIPE, int STAGES>
tg_status launch_grad_tiles(const GatedParams &p, const ProductPlan &plan, hipStream_t s) {
    hipLaunchKernelGGL((gate_grad_tile_kernel<C, P, B_KS, PIPE, STAGES>), dim3((unsigned)plan.gx), dim3(C::THREADS), 0, s, p);
    return launched();
}

template <int DT, bool TRANS>
tg_status launch_gate_grad_as(const GatedParams &p, hipStream_t s) {
    const ProductPlan plan = plan_gate_grad_as<DT, TRANS>(p.experts, p.rows, p.N, p.K);
    if (!plan.fits()) return TG_ERR_UNSUPPORTED;
    if (plan.info.kernel == TG_EXPERTS_STREAM) {
        const unsigned lds = plan.info.waves * StreamShape<DT, TRANS>::FRAGS * 1024;
        hipLaunchKernelGGL((gate_grad_few_kernel<DT, TRANS>), dim3((unsigned)plan.gx, plan.gy, plan.gz),
                           dim3(64 * plan.info.waves), lds, s, p);
        return launched();
    }
    if (plan.info.tile_m == 256) return launch_grad_tiles<Tile256<DT>, Tile128<DT>, !TRANS, true, 4>(p, plan, s);
    if constexpr (DT == DT_F32) {
        return launch_grad_tiles<Tile64<DT>, Tile64<DT>, !TRANS, true, 4>(p, plan, s);
    } else {
        if (plan.info.tile_n == 128) return launch_grad_tiles<Tile64x128<DT>, Tile64x128<DT>, !TRANS, false, 4>(p, plan, s);
        return launch_grad_tiles<Tile64<DT>, Tile64<DT>, !TRANS, false, 4>(p, plan, s);
    }
}

}  // namespace

template <int DT>
tg_status launch_gated(const GatedParams &p, bool transposed, void *workspace, hipStream_t s) {
    return transposed ? launch_gated_as<DT, true>(p, workspace, s) : launch_gated_as<DT, false>(p, workspace, s);
}

template <int DT>
tg_status launch_gate_grad(const GatedParams &p, bool transposed, hipStream_t s) {
    return transposed ? launch_gate_grad_as<DT, true>(p, s) : launch_gate_grad_as<DT, false>(p, s);
}

template <int DT>
tg_status launch_gate(const GatedParams &p, bool grad, hipStream_t s) {
    const int64_t blocks = cdiv((int64_t)p.rows * cdiv(p.N, Chunk<DT>::PER), 256);
    if (blocks > kGridX * 65535) return TG_ERR_UNSUPPORTED;
    if (grad) hipLaunchKernelGGL((gate_kernel<DT, true>), wide_grid(blocks), dim3(256), 0, s, p);
    else hipLaunchKernelGGL((gate_kernel<DT, false>), wide_grid(blocks), dim3(256), 0, s, p);
    return launched();
}

}  // namespace tg
