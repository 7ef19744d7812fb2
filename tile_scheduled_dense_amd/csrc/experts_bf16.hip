// experts_bf16.hip -- the bf16 kernels of the expert products (experts.hpp).
#include "experts_kernels.hpp"

namespace tg {

template tg_status launch_grouped<DT_BF16>(const GroupedParams &p, bool transposed, hipStream_t s);
template tg_status launch_wgrad<DT_BF16>(const GroupedParams &p, hipStream_t s);
template tg_status launch_q4<DT_BF16>(const Q4Params &p, int group, hipStream_t s);

}  // namespace tg
