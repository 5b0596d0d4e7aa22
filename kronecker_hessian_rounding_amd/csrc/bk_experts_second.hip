// bk_experts_second.hip -- the experts' second product, of rows in pieces (kernels in bk_experts.hpp).
#include "bk_experts.hpp"

namespace bk {
template void launch_experts_second<kH2>(const ExpertArgs&, int, int, int, hipStream_t);
template void launch_experts_second<kH3>(const ExpertArgs&, int, int, int, hipStream_t);
template void launch_experts_second_few<2>(const FewArgs&, int, int, int, void*, int, int64_t, hipStream_t);
template void launch_experts_second_few<3>(const FewArgs&, int, int, int, void*, int, int64_t, hipStream_t);
}  // namespace bk
