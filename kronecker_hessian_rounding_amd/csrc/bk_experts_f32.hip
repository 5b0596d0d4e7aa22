// bk_experts_f32.hip -- the experts' first product of f32 token rows (kernels in bk_experts.hpp).
#include "bk_experts.hpp"

namespace bk {
template void launch_experts_first<kF32>(const ExpertArgs&, int, int, int, hipStream_t);
template void launch_experts_first_few<kF32>(const FewArgs&, int, int, hipStream_t);
}  // namespace bk
