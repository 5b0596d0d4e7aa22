// bk_experts_e4m3.hip -- the experts' first product of e4m3 token rows (kernels in bk_experts.hpp).
#include "bk_experts.hpp"

namespace bk {
template void launch_experts_first<kF8>(const ExpertArgs&, int, int, int, hipStream_t);
template void launch_experts_first_few<kF8>(const FewArgs&, int, int, hipStream_t);
}  // namespace bk
