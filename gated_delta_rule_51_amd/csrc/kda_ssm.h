// Device helpers of the state-space scan kernels.
#pragma once

#include "kda_device.h"

namespace kda {

// softplus(z) = max(z, 0) + log(1 + u), u = e^-|z|.  The step multiplies x
// and, far below 1, is the logarithm alone, so that keeps its relative accuracy:
//     log(1 + u) = 2 atanh(s) = 2 s (1 + s^2/3 + s^4/5 + ...),  s = u / (2 + u) <= 1/3,
// to s^14 (the rest is below 2e-9 of it), and the exponent of u is kept to two
// floats.  About 30 instructions, against 140 of log1pf and expf.
__device__ __forceinline__ float softplus_f(float z) {
    const float n = -fabsf(z), t = n * kLog2e;
    const float rest = n > -200.f ? fmaf(n, kLog2e, -t) + n * 1.92596299e-8f : 0.f;   // log2(e) less kLog2e; infinite z has none
    float u = exp2f(t);   // with its subnormals: a large rate may multiply them
    u = fmaf(u, rest * 0.693147181f, u);
    const float d = 2.f + u, r = __builtin_amdgcn_rcpf(d);
    float s = u * r;
    s = fmaf(fmaf(-s, d, u), r, s);
    const float q = s * s;
    float p = 1.f / 15;
    p = fmaf(p, q, 1.f / 13);
    p = fmaf(p, q, 1.f / 11);
    p = fmaf(p, q, 1.f / 9);
    p = fmaf(p, q, 1.f / 7);
    p = fmaf(p, q, 1.f / 5);
    p = fmaf(p, q, 1.f / 3);
    s += s;
    return fmaxf(z, 0.f) + fmaf(s * q, p, s);
}

// Two floats rounded to bf16 in one instruction.
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{lo, hi}, bf16x2));
}

}  // namespace kda
