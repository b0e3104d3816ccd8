// Device helpers of the state-space scan kernels.
#pragma once

#include "kda_device.h"

namespace kda {

// softplus(z) = max(z, 0) + log(1 + e^-|z|).  The step multiplies x and, far
// below 1, is the small term alone, so it is formed with log1p: the sum
// rounded to fp32 first would lose 6e-5 of a step of 1e-3.
__device__ __forceinline__ float softplus_f(float z) { return fmaxf(z, 0.f) + log1pf(expf(-fabsf(z))); }

// Two floats rounded to bf16 in one instruction.
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{lo, hi}, bf16x2));
}

}  // namespace kda
