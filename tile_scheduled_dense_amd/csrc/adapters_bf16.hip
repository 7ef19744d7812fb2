// adapters_bf16.hip -- the bf16 kernels of a projection with adapters (ffn.hpp).
#include "adapters_kernels.hpp"

namespace tg {

template tg_status launch_adapters<DT_BF16>(const AdapterParams &p, bool transposed, void *workspace, hipStream_t s);
template tg_status launch_adapters_wgrad<DT_BF16>(const AdapterGradParams &p, void *workspace, hipStream_t s);

}  // namespace tg
