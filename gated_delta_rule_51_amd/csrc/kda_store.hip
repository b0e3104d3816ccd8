// Keys and values into the blocks of a paged cache, in 8 bits (OCP e4m3).
//
// A block of b tokens has one scale per head, 2^e with the least e >= -100 for
// which |x| <= 448 * 2^e over its tokens; 448 is e4m3's largest value.  A power
// of two costs a floating format nothing (the fraction is the same under any
// of them), makes x / 2^e exact, and lets a block's scale grow when a later
// token needs it: what the block holds already is multiplied by 2^(old - new),
// exactly but where a value falls below e4m3's least normal one.
//
// Tokens come with their slots; consecutive tokens on consecutive slots of one
// block are a run, and a run is one workgroup's work (per head, keys and values
// apart), so no two touch a block's bytes or its scale.  Bound by HBM: the rows
// once, their bytes once.
#include "kda_device.h"
#include "kda_internal.h"

namespace kda {
namespace {

constexpr int kThreads = 256;

template <typename T> struct Wide;   // 16 bytes of a row
template <> struct Wide<bf16> {
    static constexpr int N = 8;
    u32x4 w;
    __device__ __forceinline__ float at(int i) const { return i & 1 ? __uint_as_float(w[i >> 1] & 0xffff0000u) : __uint_as_float(w[i >> 1] << 16); }
};
template <> struct Wide<float> {
    static constexpr int N = 4;
    u32x4 w;
    __device__ __forceinline__ float at(int i) const { return __uint_as_float(w[i]); }
};

// The least power of two s >= 2^-100 with x <= 448 s (x finite, >= 0):
// 448 = 1.75 * 2^8, so from x = m 2^k, m in [1, 2), s = 2^(k - 8), or twice
// that where m > 1.75.
__device__ __forceinline__ float scale_for(float x) {
    const uint32_t bits = __float_as_uint(x);
    const int k = (int)(bits >> 23) - 127 - 8 + ((bits & 0x7fffff) > 0x600000);
    return __uint_as_float((uint32_t)(max(k, -100) + 127) << 23);
}

// Four values, x * inv rounded to the nearest e4m3 (ties to even); what is not
// finite becomes NaN.
__device__ __forceinline__ float ready(float x, float inv) {
    return __builtin_fabsf(x) < __builtin_inff() ? x * inv : __builtin_nanf("");
}
__device__ __forceinline__ uint32_t pack4(float a, float b, float c, float d, float inv) {
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(ready(a, inv), ready(b, inv), 0, false);
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(ready(c, inv), ready(d, inv), w, true);
}
// Four stored values times f, those whose bit in `some` is set.
__device__ __forceinline__ uint32_t rescale4(uint32_t w, float f, uint32_t some) {
    const f32x2 a = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, false), b = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, true);
    const uint32_t y = pack4(a[0], a[1], b[0], b[1], f);
    uint32_t mask = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) mask |= some >> i & 1 ? 0xffu << (8 * i) : 0;
    return (y & mask) | (w & ~mask);
}

// Tokens [t, t + m) of one head go to offsets [f, f + m) of a block.
template <typename T, int D, bool VALUES>
__device__ __forceinline__ void store_run(const T *x, long stride, uint8_t *cache, float *scale, int f, int m, int shift,
                                          uint8_t *tile, float *most) {
    constexpr int N = Wide<T>::N, LPR = D / N, RPP = kThreads / LPR, HELD = 4;
    const int tid = threadIdx.x, c = tid % LPR, r0 = tid / LPR, bs = 1 << shift, pitch = bs + 16;
    Wide<T> held[HELD];   // the first rows stay in registers, any others are read again
    float top = 0.f;
    const auto see = [&](const Wide<T> &y) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const float z = __builtin_fabsf(y.at(i));
            top = __builtin_fmaxf(top, z < __builtin_inff() ? z : 0.f);
        }
    };
    const auto load = [&](int r) { return Wide<T>{*reinterpret_cast<const u32x4 *>(x + (long)r * stride + c * N)}; };
#pragma unroll
    for (int p = 0; p < HELD; ++p)
        if (r0 + p * RPP < m) held[p] = load(r0 + p * RPP);
#pragma unroll
    for (int p = 0; p < HELD; ++p)
        if (r0 + p * RPP < m) see(held[p]);
    for (int r = r0 + HELD * RPP; r < m; r += RPP) see(load(r));
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) top = __builtin_fmaxf(top, __shfl_xor(top, d, 64));
    if ((tid & 63) == 0) most[tid >> 6] = top;
    const float before = f ? *scale : 0.f;
    __syncthreads();
    top = __builtin_fmaxf(__builtin_fmaxf(most[0], most[1]), __builtin_fmaxf(most[2], most[3]));
    const float after = __builtin_fmaxf(scale_for(top), before), inv = 1.f / after, again = before * inv;
    const bool grown = f && after > before;
    if (tid == 0 && (grown || !f)) *scale = after;
    const auto put = [&](int r, const Wide<T> &y) {
        uint32_t w[N / 4];
#pragma unroll
        for (int i = 0; i < N / 4; ++i) w[i] = pack4(y.at(4 * i), y.at(4 * i + 1), y.at(4 * i + 2), y.at(4 * i + 3), inv);
        if constexpr (VALUES) {
#pragma unroll
            for (int i = 0; i < N; ++i) tile[(c * N + i) * pitch + f + r] = (uint8_t)(w[i / 4] >> (8 * (i & 3)));
        } else if constexpr (N == 8) {
            *reinterpret_cast<u32x2 *>(cache + (long)(f + r) * D + c * N) = u32x2{w[0], w[1]};
        } else {
            *reinterpret_cast<uint32_t *>(cache + (long)(f + r) * D + c * N) = w[0];
        }
    };
#pragma unroll
    for (int p = 0; p < HELD; ++p)
        if (r0 + p * RPP < m) put(r0 + p * RPP, held[p]);
    for (int r = r0 + HELD * RPP; r < m; r += RPP) put(r, load(r));
    if constexpr (VALUES) {
        __syncthreads();
        // sixteen tokens of one channel a thread, tokens side by side
        const int per = bs >> 4;
        for (int i = tid; i < D * per; i += kThreads) {
            const int d = i / per, from = (i % per) * 16;
            const int lo = max(f - from, 0), hi = min(f + m - from, 16);   // those of the run
            uint8_t *to = cache + (long)d * bs + from;
            const uint8_t *with = tile + d * pitch + from;
            if (lo == 0 && hi >= 16) {
                *reinterpret_cast<u32x4 *>(to) = *reinterpret_cast<const u32x4 *>(with);
            } else {
                for (int k = lo; k < hi; ++k) to[k] = with[k];
                if (grown && f > from) {
                    for (int k = 0; k < min(f - from, 16); k += 4) {
                        const uint32_t some = f - from - k >= 4 ? 0xf : (1u << (f - from - k)) - 1;
                        const uint32_t y = rescale4(*reinterpret_cast<const uint32_t *>(to + k), again, some);
                        for (int j = 0; j < 4; ++j)
                            if (some >> j & 1) to[k + j] = (uint8_t)(y >> (8 * j));
                    }
                }
            }
        }
    } else if (grown) {
        for (int i = tid; i < f * (D / 4); i += kThreads) {
            uint32_t *to = reinterpret_cast<uint32_t *>(cache) + i;
            *to = rescale4(*to, again, 0xf);
        }
    }
    __syncthreads();
}

// The runs that begin among tokens [blockIdx.x * R, + R), R <= 128.
template <typename T, int D> __global__ __launch_bounds__(kThreads) void store_kernel(const StoreArgs a, int R) {
    __shared__ __align__(16) uint8_t tile[D * (128 + 16)];
    __shared__ float most[4];
    const int lane = threadIdx.x & 63, h = blockIdx.y, bs = 1 << a.block_shift, t0 = blockIdx.x * R;
    for (int half = 0; half < R; half += 64) {
        const int t = t0 + half + lane;
        const int s = half + lane < R && t < a.total_tokens ? a.slots[t] : -1;
        const bool leads = s >= 0 && (s >> a.block_shift) < a.num_blocks && ((s & (bs - 1)) == 0 || t == 0 || a.slots[t - 1] != s - 1);
        unsigned long long lead = __ballot(leads);
        while (lead) {
            const int k = __builtin_ctzll(lead);
            lead &= lead - 1;
            const int first = t0 + half + k, slot = __builtin_amdgcn_readlane(s, k), f = slot & (bs - 1), block = slot >> a.block_shift;
            int m = 0;   // tokens of the run
            for (int i = 0; i < bs; i += 64) {
                const int j = i + lane;
                const bool in = f + j < bs && first + j < a.total_tokens && a.slots[first + j] == slot + j;
                const unsigned long long out = __ballot(!in);
                m = i + (out ? __builtin_ctzll(out) : 64);
                if (out) break;
            }
            const long at = (long)block * a.heads + h;
            if (blockIdx.z)
                store_run<T, D, true>(static_cast<const T *>(a.v) + first * a.v_stride + (long)h * D, a.v_stride,
                                      a.v_cache + at * D * bs, a.v_scale + at, f, m, a.block_shift, tile, most);
            else
                store_run<T, D, false>(static_cast<const T *>(a.k) + first * a.k_stride + (long)h * D, a.k_stride,
                                       a.k_cache + at * D * bs, a.k_scale + at, f, m, a.block_shift, tile, most);
        }
    }
}

template <typename T, int D> hipError_t launch(const StoreArgs &a, int R, hipStream_t stream) {
    store_kernel<T, D><<<dim3((a.total_tokens + R - 1) / R, a.heads, 2), kThreads, 0, stream>>>(a, R);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_kv_store(const StoreArgs &a, hipStream_t stream) {
    // tokens looked at by one workgroup: one of few tokens, each of which is
    // likely to be a run, up to a block of many
    int R = 1;
    while (R < (1 << a.block_shift) && (long)a.total_tokens * a.heads / R > 4096) R *= 2;
    if (a.io_bf16) return a.d == 64 ? launch<bf16, 64>(a, R, stream) : launch<bf16, 128>(a, R, stream);
    return a.d == 64 ? launch<float, 64>(a, R, stream) : launch<float, 128>(a, R, stream);
}

}  // namespace kda
