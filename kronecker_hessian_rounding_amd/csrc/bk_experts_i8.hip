// bk_experts_i8.hip -- the experts' first product of i8 token rows (kernels in bk_experts.hpp).
#include "bk_experts.hpp"

namespace bk {
template void launch_experts_first<kI8>(const ExpertArgs&, int, int, int, hipStream_t);
template void launch_experts_first_few<kI8>(const FewArgs&, int, int, hipStream_t);
}  // namespace bk
