// bk_matvec_i8.hip -- the products of int8 token rows (kernels in bk_matvec.hpp).
#include "bk_matvec.hpp"

namespace bk {
template void launch_products<kI8>(const MvArgs&, int, int, hipStream_t);
}  // namespace bk
