// bk_matvec_f16.hip -- the products of fp16 token rows (kernels in bk_matvec.hpp).
#include "bk_matvec.hpp"

namespace bk {
template void launch_products<kF16>(const MvArgs&, int, int, hipStream_t);
}  // namespace bk
