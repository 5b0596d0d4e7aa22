// bk_experts_second.hip -- the experts' second product, of fp32 rows (kernels in bk_experts.hpp).
#include "bk_experts.hpp"

namespace bk {
template void launch_experts_second<kF32>(const ExpertArgs&, int, int, hipStream_t);
}  // namespace bk
