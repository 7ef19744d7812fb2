// gated_bf16.hip -- the bf16 kernels of the gated pair and its gradient (ffn.hpp).
#include "gated_kernels.hpp"

namespace tg {

template tg_status launch_gated<DT_BF16>(const GatedParams &p, bool transposed, void *workspace, hipStream_t s);
template tg_status launch_gate_grad<DT_BF16>(const GatedParams &p, bool transposed, hipStream_t s);
template tg_status launch_gate<DT_BF16>(const GatedParams &p, bool grad, hipStream_t s);

}  // namespace tg
