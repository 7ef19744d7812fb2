// experts.hpp -- the expert products' kernels of each input type, launched on a
// stream; one translation unit per type (experts_bf16.hip, experts_f16.hip,
// experts_f32.hip), which the build compiles in parallel.  Arguments have been
// checked by the C ABI (experts.hip).
#pragma once

#include <hip/hip_runtime.h>

#include "grouped_ring.hpp"
#include "q4.hpp"
#include "tile_gemm.h"

namespace tg {

template <int DT> tg_status launch_grouped(const GroupedParams &p, bool transposed, hipStream_t s);
template <int DT> tg_status launch_wgrad(const GroupedParams &p, hipStream_t s);
template <int DT> tg_status launch_q4(const Q4Params &p, int group, hipStream_t s);

}  // namespace tg
