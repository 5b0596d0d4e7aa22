// bk_matvec_e4m3.hip -- the products of e4m3 token rows (kernels in bk_matvec.hpp).
#include "bk_matvec.hpp"

namespace bk {
template void launch_products<kF8>(const MvArgs&, int, int, hipStream_t);
}  // namespace bk
