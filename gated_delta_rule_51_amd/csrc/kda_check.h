// Checks of host-visible arguments shared by the C entry points.
#pragma once

#include <hip/hip_runtime.h>

#include "../../include/kda.h"

namespace kda {

inline bool dim_ok(int d) { return d == 32 || d == 64 || d == 128; }
inline bool dtype_ok(int t) { return t == KDA_F32 || t == KDA_BF16; }
inline bool gate_ok(int t) { return t == KDA_GATE_CHANNEL || t == KDA_GATE_SCALAR; }
inline bool aligned(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline size_t io_size(int t) { return t == KDA_BF16 ? 2 : 4; }

// Byte ranges [p, p + n) overlap?
inline bool overlap(const void *a, size_t na, const void *b, size_t nb) {
    if (!a || !b || na == 0 || nb == 0) return false;
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x < y + nb && y < x + na;
}

inline kda_status hip_status(hipError_t e) { return e == hipSuccess ? KDA_OK : KDA_ERR_HIP; }

}  // namespace kda
