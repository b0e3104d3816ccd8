// Device helpers shared by the libkda kernels (gfx950 only).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace kda {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

// bf16 is carried as raw 16-bit storage; conversions are explicit.
struct bf16 {
    uint16_t bits;
};

__device__ __forceinline__ float bf16_to_f32(uint16_t b) { return __uint_as_float((uint32_t)b << 16); }

// Round to nearest even (hardware v_cvt_pk_bf16_f32 on gfx950).
__device__ __forceinline__ uint16_t f32_to_bf16(float f) {
    __bf16 h = (__bf16)f;
    return __builtin_bit_cast(uint16_t, h);
}

// exp(x) through the hardware base-2 exponential.
__device__ __forceinline__ float exp_f(float x) { return __builtin_amdgcn_exp2f(x * 1.4426950408889634f); }

constexpr float kLog2e = 1.4426950408889634f;

// Gate activation from raw inputs: the decay factor exp(g) for
// g = -A softplus(z), A = exp(A_log), given zl = z log2(e) (z = x + dt_bias):
//     exp(g) = 2^(-A sp),  sp = softplus(z) log2(e) = max(zl, 0) + log2(1 + 2^-|zl|).
// Three hardware transcendentals.  log2 of the rounded 1 + 2^-|zl| costs at
// most ~1e-7 of sp in absolute terms (relative accuracy is lost only where sp
// itself is tiny), i.e. |error of g| <= ~1e-7 A: far below the rounding of a
// bf16 x (2^-9 relative).
__device__ __forceinline__ float gate_decay(float zl, float A) {
    const float sp = __builtin_fmaxf(zl, 0.f) +
                     __builtin_amdgcn_logf(1.f + __builtin_amdgcn_exp2f(-__builtin_fabsf(zl)));
    return __builtin_amdgcn_exp2f(-A * sp);
}

// beta = sigmoid(b) = 1 / (1 + e^-b); e^-b overflowing to +inf gives 0.
__device__ __forceinline__ float sigmoid_f(float b) {
    return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-b * kLog2e));
}

// Word 3 of a raw buffer resource on gfx9-family parts: 32-bit data format,
// no swizzle; untyped 16-byte accesses with a byte range check.
constexpr int kBufferWord3 = 0x00020000;

// Element type traits for io / state tensors.
template <typename T> struct io_traits;
template <> struct io_traits<float> {
    static constexpr int bytes = 4;
    __device__ static __forceinline__ float load(const float *p, long i) { return p[i]; }
    __device__ static __forceinline__ void store(float *p, long i, float x) { p[i] = x; }
};
template <> struct io_traits<bf16> {
    static constexpr int bytes = 2;
    __device__ static __forceinline__ float load(const bf16 *p, long i) { return bf16_to_f32(p[i].bits); }
    __device__ static __forceinline__ void store(bf16 *p, long i, float x) { p[i].bits = f32_to_bf16(x); }
};

// Load 4 consecutive elements as floats (16 B for f32, 8 B for bf16).
__device__ __forceinline__ f32x4 load4(const float *p) { return *reinterpret_cast<const f32x4 *>(p); }
__device__ __forceinline__ f32x4 load4(const bf16 *p) {
    u32x2 w = *reinterpret_cast<const u32x2 *>(p);
    f32x4 r;
    r[0] = __uint_as_float(w[0] << 16);
    r[1] = __uint_as_float(w[0] & 0xffff0000u);
    r[2] = __uint_as_float(w[1] << 16);
    r[3] = __uint_as_float(w[1] & 0xffff0000u);
    return r;
}

__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
    return (uint32_t)f32_to_bf16(lo) | ((uint32_t)f32_to_bf16(hi) << 16);
}

// The sequence whose tiles of R tokens hold `slot`, where sequence n's tiles
// take the slots floor(cu[n] / R) + n onwards: at least ceil(L / R) of them lie
// before the next sequence's first (one where L is 0), so cu_seqlens alone
// tells what a slot stands for, and floor(T / R) + N slots hold every tile.
// With FIRST 0 the tiles after each sequence's first take the slots
// floor(cu[n] / R) onwards, floor(T / R) in all.  The whole wave searches, 64
// ways a step.
template <int FIRST = 1> __device__ __forceinline__ int slot_sequence(const int32_t *cu, int num_seqs, int slot, int R) {
    const int lane = threadIdx.x & 63;
    int lo = 0, n = num_seqs;
    while (n > 1) {
        const int step = (n + 63) / 64, i = lane * step;
        const unsigned long long m = __ballot(i < n && cu[lo + min(i, n - 1)] / R + FIRST * (lo + i) <= slot);
        const int k = (63 - __builtin_clzll(m | 1)) * step;
        lo += k;
        n = min(step, n - k);
    }
    return lo;
}

// Inclusive sums over the wave's lanes, without a trip through LDS.
template <int CTRL, int ROWS> __device__ __forceinline__ double dpp_add(double x) {
    const u32x2 w = __builtin_bit_cast(u32x2, x);
    return x + __builtin_bit_cast(double, u32x2{(uint32_t)__builtin_amdgcn_update_dpp(0, (int)w[0], CTRL, ROWS, 0xf, false),
                                                (uint32_t)__builtin_amdgcn_update_dpp(0, (int)w[1], CTRL, ROWS, 0xf, false)});
}
__device__ __forceinline__ double wave_scan(double x) {
    x = dpp_add<0x111, 0xf>(x);   // from 1, 2, 4 and 8 lanes below within a row of 16
    x = dpp_add<0x112, 0xf>(x);
    x = dpp_add<0x114, 0xf>(x);
    x = dpp_add<0x118, 0xf>(x);
    x = dpp_add<0x142, 0xa>(x);   // a row's last lane to the next row
    return dpp_add<0x143, 0xc>(x);   // lane 31 to the upper half
}
__device__ __forceinline__ double lane_value(double x, int lane) {
    const u32x2 w = __builtin_bit_cast(u32x2, x);
    return __builtin_bit_cast(double, u32x2{(uint32_t)__builtin_amdgcn_readlane((int)w[0], lane),
                                            (uint32_t)__builtin_amdgcn_readlane((int)w[1], lane)});
}

template <int W> __device__ __forceinline__ float group_sum(float x) {
    // Sum over W consecutive lanes (W a power of two <= 64).
#pragma unroll
    for (int m = W / 2; m >= 1; m >>= 1) x += __shfl_xor(x, m, 64);
    return x;
}

}  // namespace kda
