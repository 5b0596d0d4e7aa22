// bk_matvec_f32.hip -- the products of fp32 token rows (kernels in bk_matvec.hpp).
#include "bk_matvec.hpp"

namespace bk {
template void launch_products<kF32>(const MvArgs&, int, int, hipStream_t);
}  // namespace bk
