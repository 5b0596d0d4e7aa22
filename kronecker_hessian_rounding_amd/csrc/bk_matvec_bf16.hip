// bk_matvec_bf16.hip -- the products of bf16 token rows (kernels in bk_matvec.hpp).
#include "bk_matvec.hpp"

namespace bk {
template void launch_products<kBF16>(const MvArgs&, int, int, hipStream_t);
}  // namespace bk
