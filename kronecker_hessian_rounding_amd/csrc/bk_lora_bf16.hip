// bk_lora_bf16.hip -- low-rank adapters in bf16 (kernels in bk_lora.hpp).
#include "bk_lora.hpp"

namespace bk {
template void launch_lora_adapters<__bf16>(const LoraArgs&, int, hipStream_t);
}  // namespace bk
