// bk_lora_f32.hip -- low-rank adapters in fp32 (kernels in bk_lora.hpp).
#include "bk_lora.hpp"

namespace bk {
template void launch_lora_adapters<float>(const LoraArgs&, int, hipStream_t);
}  // namespace bk
