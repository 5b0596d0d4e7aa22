// bk_lora_f16.hip -- low-rank adapters in fp16 (kernels in bk_lora.hpp).
#include "bk_lora.hpp"

namespace bk {
template void launch_lora_adapters<_Float16>(const LoraArgs&, int, hipStream_t);
}  // namespace bk
