// ffn.hpp -- the kernels of a feed-forward block's operators for each input type, launched
// on a stream; one translation unit per operator and type, which the build compiles in
// parallel.  Arguments have been checked by the C ABI (ffn.hip).
#pragma once

#include <hip/hip_runtime.h>

#include "adapters.hpp"
#include "tile_gemm.h"

namespace tg {

// workspace: NULL where there is none of the plan's size
template <int DT> tg_status launch_gated(const GatedParams &p, bool transposed, void *workspace, hipStream_t s);
template <int DT> tg_status launch_gate_grad(const GatedParams &p, bool transposed, hipStream_t s);
template <int DT> tg_status launch_gate(const GatedParams &p, bool grad, hipStream_t s);
template <int DT> tg_status launch_adapters(const AdapterParams &p, bool transposed, void *workspace, hipStream_t s);
template <int DT> tg_status launch_adapters_wgrad(const AdapterGradParams &p, void *workspace, hipStream_t s);

}  // namespace tg
