// bk_experts_second.hip -- the experts' second product, of fp32 rows and of pieces (kernels in bk_experts.hpp).
#include "bk_experts.hpp"

namespace bk {
template void launch_experts_second<kF32>(const ExpertArgs&, int, int, hipStream_t);
template void launch_experts_second_few<2>(const FewArgs&, int, int, int, void*, int, int64_t, hipStream_t);
template void launch_experts_second_few<3>(const FewArgs&, int, int, int, void*, int, int64_t, hipStream_t);
}  // namespace bk
