// bk_experts_bf16.hip -- the experts' first product of bf16 token rows (kernels in bk_experts.hpp).
#include "bk_experts.hpp"

namespace bk {
template void launch_experts_first<kBF16>(const ExpertArgs&, int, int, int, hipStream_t);
template void launch_experts_first_few<kBF16>(const FewArgs&, int, int, hipStream_t);
}  // namespace bk
