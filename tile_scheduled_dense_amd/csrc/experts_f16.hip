// experts_f16.hip -- the f16 kernels of the expert products (experts.hpp).
#include "experts_kernels.hpp"

namespace tg {

template tg_status launch_grouped<DT_F16>(const GroupedParams &p, bool transposed, hipStream_t s);
template tg_status launch_wgrad<DT_F16>(const GroupedParams &p, hipStream_t s);
template tg_status launch_q4<DT_F16>(const Q4Params &p, int group, hipStream_t s);

}  // namespace tg
