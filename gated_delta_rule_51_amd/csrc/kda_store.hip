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
// block are a run, and a run is one workgroup's work, or one wave's (per head, keys
// and values apart), so no two touch a block's bytes or its scale.  Bound by HBM: the
// rows once, their bytes once (35,100 tokens x 8 heads x 128, bf16: 216 MB in 57 us,
// 3.8 TB/s, where a copy reaches 4.8); single tokens by latency (256 tokens 5.4 us).
#include <algorithm>

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

// Four values, x * inv rounded to the nearest e4m3 (ties to even).  None is above
// 448 but infinities, which become NaN, as e4m3 has none.
__device__ __forceinline__ uint32_t pack4(float a, float b, float c, float d, float inv) {
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(a * inv, b * inv, 0, false);
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c * inv, d * inv, w, true);
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

// Where values of a block's tile lie in LDS: channel d's tokens 16 p .. + 15, whole,
// turned by d / 8 so that neither the words written nor the 16 bytes read meet in
// a bank more than four times.
__device__ __forceinline__ int tile_at(int d, int p, int shift) {
    return (d << shift) + 16 * ((p + (d >> 3)) & ((1 << (shift - 4)) - 1));
}

// One head's scale of a block, f tokens of which it holds already: after a run
// with the largest value `top`.
struct Scale { float after, inv, again; bool grown; };
__device__ __forceinline__ Scale scale_after(float top, float before, int f) {
    Scale s;
    s.after = __builtin_fmaxf(scale_for(top), f ? before : 0.f);
    s.inv = 1.f / s.after;
    s.again = before * s.inv;
    s.grown = f && s.after > before;
    return s;
}

template <typename T> __device__ __forceinline__ float top_of(const Wide<T> &y, float top) {
#pragma unroll
    for (int i = 0; i < Wide<T>::N; ++i) {
        const float z = __builtin_fabsf(y.at(i));
        top = __builtin_fmaxf(top, z < __builtin_inff() ? z : 0.f);
    }
    return top;
}
template <typename T> __device__ __forceinline__ void put_row(uint8_t *to, const Wide<T> &y, float inv) {
    uint32_t w[Wide<T>::N / 4];
#pragma unroll
    for (int i = 0; i < Wide<T>::N / 4; ++i) w[i] = pack4(y.at(4 * i), y.at(4 * i + 1), y.at(4 * i + 2), y.at(4 * i + 3), inv);
    if constexpr (Wide<T>::N == 8) *reinterpret_cast<u32x2 *>(to) = u32x2{w[0], w[1]};
    else *reinterpret_cast<uint32_t *>(to) = w[0];
}

// The first f tokens of a block stored again, by `threads` threads of number i.
// Keys [b, D]; values [D, b].
template <int D> __device__ __forceinline__ void again_keys(uint8_t *cache, int f, float again, int i, int threads) {
    for (; i < f * (D / 4); i += threads) {
        uint32_t *to = reinterpret_cast<uint32_t *>(cache) + i;
        *to = rescale4(*to, again, 0xf);
    }
}
template <int D> __device__ __forceinline__ void again_values(uint8_t *cache, int f, int shift, float again, int i, int threads) {
    const int words = (f + 3) / 4;
    for (; i < D * words; i += threads) {
        const int d = i / words, k = i % words * 4;
        uint8_t *to = cache + (d << shift) + k;
        const uint32_t some = f - k >= 4 ? 0xf : (1u << (f - k)) - 1;
        const uint32_t y = rescale4(*reinterpret_cast<const uint32_t *>(to), again, some);
        for (int j = 0; j < 4; ++j)   // those behind f may be another's to write
            if (some >> j & 1) to[j] = (uint8_t)(y >> (8 * j));
    }
}

// A run of up to kShort tokens: a head's row, keys or values, is LPR lanes' work, so
// one workgroup stores a token's 2 H rows without a barrier.
constexpr int kShort = 4;
template <typename T, int D>
__device__ __forceinline__ void store_short(const StoreArgs &a, int first, int f, int m, int block, int unit0, int units) {
    constexpr int N = Wide<T>::N, LPR = D / N;
    int tid = threadIdx.x;
    asm volatile("" : "+v"(tid));
    const int c = tid % LPR, shift = a.block_shift;
    const int unit = unit0 + tid / LPR;
    if (unit >= units) return;
    const bool values = unit >= a.heads;
    const int h = values ? unit - a.heads : unit;
    const long at = (long)block * a.heads + h, stride = values ? a.v_stride : a.k_stride;
    const T *x = static_cast<const T *>(values ? a.v : a.k) + first * stride + (long)h * D + c * N;
    float *scale = (values ? a.v_scale : a.k_scale) + at;
    uint8_t *cache = (values ? a.v_cache : a.k_cache) + ((at * D) << shift);
    Wide<T> y[kShort];
    float top = 0.f;
    const float before = f ? *scale : 0.f;
#pragma unroll
    for (int r = 0; r < kShort; ++r) y[r] = Wide<T>{*reinterpret_cast<const u32x4 *>(x + min(r, m - 1) * stride)};
#pragma unroll
    for (int r = 0; r < kShort; ++r) top = top_of(y[r], top);   // the last row again does no harm
#pragma unroll
    for (int d = LPR / 2; d >= 1; d >>= 1) top = __builtin_fmaxf(top, __shfl_xor(top, d, 64));
    const Scale s = scale_after(top, before, f);
    if (c == 0 && (s.grown || !f)) *scale = s.after;
    if (s.grown) {
        if (values) again_values<D>(cache, f, shift, s.again, c, LPR);
        else again_keys<D>(cache, f, s.again, c, LPR);
    }
#pragma unroll
    for (int r = 0; r < kShort; ++r) {
        if (r >= m) break;
        if (!values) {
            put_row(cache + (long)(f + r) * D + c * N, y[r], s.inv);
        } else {
#pragma unroll
            for (int i = 0; i < N; i += 4) {
                const uint32_t w = pack4(y[r].at(i), y[r].at(i + 1), y[r].at(i + 2), y[r].at(i + 3), s.inv);
#pragma unroll
                for (int e = 0; e < 4; ++e) cache[((c * N + i + e) << shift) + f + r] = (uint8_t)(w >> (8 * e));
            }
        }
    }
}

// A run of m tokens of one head, keys or values, goes to offsets [f, f + m) of a
// block.  A thread takes four tokens side by side: a word of a channel's values.
template <typename T, int D, bool VALUES>
__device__ __forceinline__ void store_run(const T *x, long stride, uint8_t *cache, float *scale, int f, int m, int shift,
                                          uint8_t *tile, float *most) {
    constexpr int N = Wide<T>::N, LPR = D / N, RPP = 4 * kThreads / LPR;
    int tid = threadIdx.x;
    asm volatile("" : "+v"(tid));   // addresses are formed here, not kept from before the loops around this
    const int c = tid % LPR, r0 = 4 * (tid / LPR);
    Wide<T> held[4];   // the first rows stay in registers, any others are read again
    float top = 0.f;
    const auto load = [&](int r) { return Wide<T>{*reinterpret_cast<const u32x4 *>(x + (long)min(r, m - 1) * stride + c * N)}; };
#pragma unroll
    for (int p = 0; p < 4; ++p) held[p] = load(r0 + p);
    const float before = f ? *scale : 0.f;
#pragma unroll
    for (int p = 0; p < 4; ++p) top = top_of(held[p], top);
    for (int r = r0 + RPP; r < m; r += RPP)
#pragma unroll
        for (int p = 0; p < 4; ++p) top = top_of(load(r + p), top);
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) top = __builtin_fmaxf(top, __shfl_xor(top, d, 64));
    if ((tid & 63) == 0) most[tid >> 6] = top;
    __syncthreads();
    top = __builtin_fmaxf(__builtin_fmaxf(most[0], most[1]), __builtin_fmaxf(most[2], most[3]));
    const Scale s = scale_after(top, before, f);
    if (tid == 0 && (s.grown || !f)) *scale = s.after;
    const auto put = [&](int r, const Wide<T> (&y)[4]) {
        if constexpr (VALUES) {
            if (r < m) {
#pragma unroll
                for (int i = 0; i < N; ++i)
                    *reinterpret_cast<uint32_t *>(tile + tile_at(c * N + i, r >> 4, shift) + (r & 15)) =
                        pack4(y[0].at(i), y[1].at(i), y[2].at(i), y[3].at(i), s.inv);
            }
        } else {
#pragma unroll
            for (int p = 0; p < 4; ++p)
                if (r + p < m) put_row(cache + (long)(f + r + p) * D + c * N, y[p], s.inv);
        }
    };
    put(r0, held);
    for (int r = r0 + RPP; r < m; r += RPP) {
#pragma unroll
        for (int p = 0; p < 4; ++p) held[p] = load(r + p);
        put(r, held);
    }
    if constexpr (VALUES) {
        __syncthreads();
        // sixteen tokens of one channel a thread, tokens side by side
        const int per = 1 << (shift - 4);
        for (int i = tid; i < D * per; i += kThreads) {
            const int d = i >> (shift - 4), from = (i & (per - 1)) * 16;
            const int lo = max(f - from, 0), hi = min(f + m - from, 16);   // those of the run
            uint8_t *to = cache + (d << shift) + from;
            if (lo == 0 && hi >= 16 && (f & 15) == 0) {
                *reinterpret_cast<u32x4 *>(to) = *reinterpret_cast<const u32x4 *>(tile + tile_at(d, (from - f) >> 4, shift));
            } else {
                for (int k = lo; k < hi; ++k) {
                    const int r = from - f + k;
                    to[k] = tile[tile_at(d, r >> 4, shift) + (r & 15)];
                }
            }
        }
        if (s.grown) again_values<D>(cache, f, shift, s.again, tid, kThreads);
    } else if (s.grown) {
        again_keys<D>(cache, f, s.again, tid, kThreads);
    }
    __syncthreads();
}

// The runs that begin among R <= 128 tokens; of their 2 H rows (H of keys, then H
// of values) those of this workgroup's turn.  Turns, not tokens, lie far apart:
// where runs are short the first turn does it all and the others only end.
template <typename T, int D> __global__ __launch_bounds__(kThreads, 8) void store_kernel(const StoreArgs a, int R, int turns) {
    __shared__ __align__(16) uint8_t tile[D * 128];
    __shared__ float most[4];
    constexpr int LPR = D / Wide<T>::N, AT_ONCE = kThreads / LPR;
    const int lane = threadIdx.x & 63, bs = 1 << a.block_shift, units = 2 * a.heads;
    const int tiles = gridDim.x / turns, turn = blockIdx.x / tiles, t0 = blockIdx.x % tiles * R;
    // a run may end in the 128 tokens behind the last it may begin with
    unsigned long long follows[4], leads[2];   // tokens on the slot behind the one before, in its block; first ones of runs
    int edge = t0 ? a.slots[t0 - 1] : -2;
    const int more = R > 64 ? 4 : bs > 64 ? 3 : 2;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const uint32_t t = (uint32_t)t0 + 64 * q + lane;   // may pass 2^31
        const int s = q < more && t < (uint32_t)a.total_tokens ? a.slots[t] : -1;
        const int up = __shfl_up(s, 1, 64), before = lane ? up : edge;
        edge = __builtin_amdgcn_readlane(s, 63);
        follows[q] = __ballot(s >= 0 && (s & (bs - 1)) && before == s - 1);
        if (q < 2) leads[q] = __ballot(64 * q + lane < R && s >= 0 && (s >> a.block_shift) < a.num_blocks) & ~follows[q];
    }
#pragma unroll 1
    for (int half = 0; half < 2; ++half) {
        unsigned long long lead = half ? leads[1] : leads[0];
#pragma unroll 1
        while (lead) {
            const int k = __builtin_ctzll(lead);
            lead &= lead - 1;
            const int first = t0 + 64 * half + k, slot = a.slots[first], f = slot & (bs - 1), block = slot >> a.block_shift;
            // tokens of the run: those that follow, without a gap
            const unsigned long long f0 = half ? follows[1] : follows[0], f1 = half ? follows[2] : follows[1], f2 = half ? follows[3] : follows[2];
            int m = 64 - k;
            if (const unsigned long long gap = ~f0 & (~1ull << k)) m = __builtin_ctzll(gap) - k;
            else if (~f1) m += __builtin_ctzll(~f1);
            else m += 64 + (~f2 ? __builtin_ctzll(~f2) : 64);
            if (m <= kShort) {
                for (int u = turn * AT_ONCE; u < units; u += turns * AT_ONCE) store_short<T, D>(a, first, f, m, block, u, units);
                continue;
            }
#pragma unroll 1
            for (int u = turn; u < units; u += turns) {
                const int h = u < a.heads ? u : u - a.heads;
                const long at = (long)block * a.heads + h;
                if (u < a.heads)
                    store_run<T, D, false>(static_cast<const T *>(a.k) + first * a.k_stride + (long)h * D, a.k_stride,
                                           a.k_cache + at * D * bs, a.k_scale + at, f, m, a.block_shift, tile, most);
                else
                    store_run<T, D, true>(static_cast<const T *>(a.v) + first * a.v_stride + (long)h * D, a.v_stride,
                                          a.v_cache + at * D * bs, a.v_scale + at, f, m, a.block_shift, tile, most);
            }
        }
    }
}

template <typename T, int D> hipError_t launch(const StoreArgs &a, int R, int turns, hipStream_t stream) {
    store_kernel<T, D><<<(unsigned)((a.total_tokens + R - 1) / R * turns), kThreads, 0, stream>>>(a, R, turns);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_kv_store(const StoreArgs &a, hipStream_t stream) {
    // Workgroups that share a run's rows, in turns: a single token is stored by the
    // first alone, so four where there are few tokens (295 tokens of runs up to 4 over
    // 16 heads: 12 us, 13.6 with a turn for each row; 1637 tokens of 7 prompts: 24 and
    // 18).  Tokens looked at by one workgroup: one of few, up to a block of many, as
    // starting a workgroup costs what looking at a token does (1731 tokens over 2
    // heads: 6.9 us with 4 tokens each, 13 with one).
    const int some = std::min(a.total_tokens <= 512 ? 4 : 65535, 2 * a.heads);
    int R = 1;
    const auto tiles = [&] { return ((long)a.total_tokens + R - 1) / R; };
    while (R < (1 << a.block_shift) && (tiles() > 512 || tiles() * some > 4096)) R *= 2;
    const long most = UINT32_MAX / kThreads / tiles();   // a grid's threads are 32 bits
    if (most < 1) return hipErrorInvalidConfiguration;
    const int turns = (int)std::min<long>(some, most);
    if (a.io_bf16) return a.d == 64 ? launch<bf16, 64>(a, R, turns, stream) : launch<bf16, 128>(a, R, turns, stream);
    return a.d == 64 ? launch<float, 64>(a, R, turns, stream) : launch<float, 128>(a, R, turns, stream);
}

}  // namespace kda
