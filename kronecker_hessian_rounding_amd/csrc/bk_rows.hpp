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

// Stores the first `count` of 4 values as elements i ..; no alignment beyond the element's is needed.
typedef float f4 __attribute__((ext_vector_type(4)));
__device__ __forceinline__ void store4(void* p, int type, int64_t i, f4 v, int count) {
    if (count < 4) {
        for (int e = 0; e < count; ++e) store_elem(p, type, i + e, e == 0 ? v[0] : e == 1 ? v[1] : v[2]);
    } else if (type == BAKRON_F32) {
        __builtin_memcpy((float*)p + i, &v, 16);
    } else if (type == BAKRON_F16) {
        typedef _Float16 h4 __attribute__((ext_vector_type(4)));
        const h4 w = {(_Float16)v[0], (_Float16)v[1], (_Float16)v[2], (_Float16)v[3]};
        __builtin_memcpy((_Float16*)p + i, &w, 8);
    } else {
        typedef __bf16 b4 __attribute__((ext_vector_type(4)));
        const b4 w = {(__bf16)v[0], (__bf16)v[1], (__bf16)v[2], (__bf16)v[3]};
        __builtin_memcpy((__bf16*)p + i, &w, 8);
    }
}

__device__ __forceinline__ float load_elem(const void* p, int type, int64_t i) {
    if (type == BAKRON_F32) return ((const float*)p)[i];
    if (type == BAKRON_F16) return (float)((const _Float16*)p)[i];
    return (float)((const __bf16*)p)[i];
}

}  // namespace bk
