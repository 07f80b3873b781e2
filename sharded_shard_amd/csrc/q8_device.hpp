// Device code that both of the 8-bit matrices' sources use.
#pragma once

#include <cstdint>

namespace fsdp {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

// Two as bf16, to nearest even, by the instruction.
__device__ __forceinline__ uint32_t two_bf16(float lo, float hi) {
    typedef float f32x2 __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{lo, hi}, bf16x2));
}

}  // namespace fsdp
