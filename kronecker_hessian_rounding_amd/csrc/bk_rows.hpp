// bk_rows.hpp -- element types of token rows: loads and stores by type, on the device.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/bakron.h"

namespace bk {

// Stores v, rounded once (to nearest even), as element i of an array of `type` (fp32, fp16 or bf16).
__device__ __forceinline__ void store_elem(void* p, int type, int64_t i, float v) {
    if (type == BAKRON_F32) ((float*)p)[i] = v;
    else if (type == BAKRON_F16) ((_Float16*)p)[i] = (_Float16)v;
    else ((__bf16*)p)[i] = (__bf16)v;
}

__device__ __forceinline__ float load_elem(const void* p, int type, int64_t i) {
    if (type == BAKRON_F32) return ((const float*)p)[i];
    if (type == BAKRON_F16) return (float)((const _Float16*)p)[i];
    return (float)((const __bf16*)p)[i];
}

}  // namespace bk
