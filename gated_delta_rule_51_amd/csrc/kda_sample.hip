// The next token of given random numbers under temperature, top-k, top-p and
// min-p, and the probabilities it is drawn from.
//
// With the logits in order (largest first, equal ones by index) each of the
// three limits keeps a beginning of that order, so together they keep
// everything up to one place of it, the cut, a pair (key, index).  The weights
// are w = exp((x - max) / T); the token is the first index with
// cum_i > u * cum_{V-1} over the weights kept.
//
// Weights are formed in 64 bits and summed as whole multiples of 2^-B (B = 46
// up to 65,536 logits, one less for every doubling): such sums do not depend on
// their order, so histograms may be filled by atomics and a token is the same
// from call to call.  A weight below 2^-(B + 1) of the largest weighs nothing.
//
// One workgroup a row.  A histogram over (max - x) / T, which is monotone, says
// in which bin a cut lies; that bin's few logits are gathered and the cut found
// among them digit by digit.  The draw narrows down from sixteenths of the row.
#include <type_traits>

#include "kda_device.h"
#include "kda_internal.h"

namespace kda {
namespace {

constexpr int kThreads = 1024, kWaves = kThreads / 64;
constexpr int kBins = 2048, kList = 4096;
constexpr float kBinsPerUnit = 64.f;   // bins of 1 / 64: the last begins at a weight of e^-32
typedef unsigned long long u64;

__device__ __forceinline__ float value(const float *p, long i) { return p[i]; }
__device__ __forceinline__ float value(const bf16 *p, long i) { return bf16_to_f32(p[i].bits); }

struct Shared {
    uint32_t count[kBins];
    u64 mass[kBins];
    u64 list[kList];
    double root[64];        // 2^(j / 64)
    uint32_t digit[256];
    u64 digit_mass[256];
    u64 sums[kWaves];
    uint32_t parts[kWaves];
    u64 out[4];
    int listed;
};

// What a row's weights come from.
struct Row {
    float top, bins;        // the largest logit; bins of one unit of logits
    double rate;            // 64 log2(e) / T
    double one;             // 2^B
    const double *root;

    __device__ __forceinline__ int bin(float x) const {
        const float z = (top - x) * bins;
        return z < (float)(kBins - 1) ? (int)z : z >= 0.f ? kBins - 1 : 0;
    }
    // 2^B exp((x - top) / T), rounded to a whole number: 2^(k / 64) from a table
    // and e^r, |r| <= ln 2 / 128, to r^5 (the rest is below 4e-17).
    __device__ __forceinline__ double real(float x) const {
        if (x == top) return one;
        const double z = ((double)x - (double)top) * rate;
        if (!(z > -64.0 * 64.0)) return 0.0;
        const double k = __builtin_rint(z), r = (z - k) * 0.010830424696249145;   // ln 2 / 64
        const int n = (int)k;
        double y = __builtin_fma(r, 1.0 / 120.0, 1.0 / 24.0);
        y = __builtin_fma(r, y, 1.0 / 6.0);
        y = __builtin_fma(r, y, 0.5);
        y = __builtin_fma(r, y, 1.0);
        y = __builtin_fma(r, y, 1.0);
        return __builtin_amdgcn_ldexp(y * root[n & 63], n >> 6) * one;
    }
    __device__ __forceinline__ u64 weight(float x) const {
        return (u64)__builtin_bit_cast(long long, real(x) + 4503599627370496.0) & 0xfffffffffffffull;   // 2^52: the fraction is the number
    }
};

// Place in the order: smaller is earlier.  The key's bits lie at the top, 32 of
// them (16 for bf16), the index below.
template <typename T> __device__ __forceinline__ u64 place_of(float x, int i) {
    const uint32_t b = x == 0.f ? 0 : __float_as_uint(x);
    const uint32_t up = b >> 31 ? b : ~b & 0x7fffffffu;   // falls as x rises
    if constexpr (sizeof(T) == 2) return (u64)(up >> 16) << 48 | (uint32_t)i;
    else return (u64)up << 32 | (uint32_t)i;
}

__device__ __forceinline__ u64 wave_sum(u64 x) {
#pragma unroll
    for (int m = 32; m >= 1; m >>= 1) x += __shfl_xor(x, m, 64);
    return x;
}

// The first of n numbers (n a multiple of 64) with which their running sum is
// at least `want`, by one wave; `before`: the sum up to it.  n where there is
// none.
template <typename N> __device__ __forceinline__ int first_reaching(const N *at, int n, u64 want, u64 &before) {
    const int lane = threadIdx.x & 63;
    u64 sum = 0;
    for (int i = 0; i < n; i += 64) {
        u64 incl = at[i + lane];
        const u64 own = incl;
#pragma unroll
        for (int m = 1; m < 64; m <<= 1) {
            const u64 y = __shfl_up(incl, m, 64);
            if (lane >= m) incl += y;
        }
        incl += sum;
        const u64 reach = __ballot(incl >= want);
        if (reach) {
            const int k = __builtin_ctzll(reach);
            before = __shfl(incl - own, k, 64);
            return i + k;
        }
        sum = __shfl(incl, 63, 64);
    }
    before = sum;
    return n;
}

// Among what each() goes over, the first place at which the running count (or
// sum of weights, BY_MASS) is at least `want`; `upto`: the sum of weights up to
// it and its own.
template <typename T, bool BY_MASS, typename Each>
__device__ u64 select(Shared &sh, const Row &row, const Each &each, int index_bits, u64 want, u64 &upto) {
    const int tid = threadIdx.x;
    u64 prefix = 0, mask = 0;
    upto = 0;
    int shift = 56;
    for (;;) {
        if (tid < 256) {
            sh.digit[tid] = 0;
            sh.digit_mass[tid] = 0;
        }
        __syncthreads();
        each([&](u64 place, float x) {
            if ((place & mask) == prefix) {
                const int d = (int)(place >> shift) & 255;
                atomicAdd(&sh.digit[d], 1u);
                atomicAdd(&sh.digit_mass[d], row.weight(x));
            }
        });
        __syncthreads();
        if (tid < 64) {
            u64 before;
            int d;
            if constexpr (BY_MASS) d = first_reaching(sh.digit_mass, 256, want, before);
            else d = first_reaching(sh.digit, 256, want, before);
            u64 less = 0;   // weights of the digits below
            for (int i = tid; i < d; i += 64) less += sh.digit_mass[i];
            less = wave_sum(less);
            if (tid == 0) {
                sh.out[0] = d;
                sh.out[1] = want - before;
                sh.out[2] = less;
                sh.out[3] = d < 256 ? sh.digit_mass[d] : 0;
            }
        }
        __syncthreads();
        const u64 d = sh.out[0], own = sh.out[3];
        want = sh.out[1];
        upto += sh.out[2];
        prefix |= d << shift;
        mask |= (u64)255 << shift;
        __syncthreads();
        if (shift == 0) {
            upto += own;
            return prefix;
        }
        shift -= 8;
        if (sizeof(T) == 2 && shift == 40) shift = 24;
        if (shift < 32 && shift >= index_bits) shift = (index_bits - 1) / 8 * 8;
    }
}

template <typename T> __global__ __launch_bounds__(kThreads) void sample_kernel(const SampleArgs a, int bits) {
    __shared__ Shared sh;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, V = a.vocab;
    const long n = blockIdx.x;
    const T *x = static_cast<const T *>(a.logits) + n * a.stride;
    float *probs = a.probs ? a.probs + n * V : nullptr;
    const float temperature = a.temperature ? a.temperature[n] : 1.f;
    const float nothing = -__builtin_inff();
    for (int i = tid; i < kBins; i += kThreads) {
        sh.count[i] = 0;
        sh.mass[i] = 0;
    }
    if (tid < 64) sh.root[tid] = exp2((double)tid / 64.0);

    // the largest logit, and the first index that has it
    float top = nothing;
    int at = INT32_MAX;
    for (int i = tid; i < V; i += kThreads) {
        const float y = value(x, i);
        if (y > top) {
            top = y;
            at = i;
        }
    }
#pragma unroll
    for (int m = 32; m >= 1; m >>= 1) {
        const float y = __shfl_xor(top, m, 64);
        const int j = __shfl_xor(at, m, 64);
        if (y > top || (y == top && j < at)) {
            top = y;
            at = j;
        }
    }
    if (lane == 0) {
        sh.parts[wave] = __float_as_uint(top);
        sh.sums[wave] = (uint32_t)at;
    }
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
        const float y = __uint_as_float(sh.parts[w]);
        const int j = (int)sh.sums[w];
        if (y > top || (y == top && j < at)) {
            top = y;
            at = j;
        }
    }
    __syncthreads();
    if (top == nothing || !(temperature > 0.f)) {   // no logit at all, or the largest
        if (tid == 0 && a.tokens) a.tokens[n] = top == nothing ? -1 : at;
        if (probs)
            for (int i = tid; i < V; i += kThreads) probs[i] = top != nothing && i == at ? 1.f : 0.f;
        return;
    }

    Row row;
    row.top = top;
    row.bins = kBinsPerUnit / temperature;
    row.rate = 64.0 * 1.4426950408889634074 / (double)temperature;
    row.one = (double)(1ull << bits);
    row.root = sh.root;
    const int index_bits = 32 - __builtin_clz(max(V - 1, 1));
    const float top_p = a.top_p ? a.top_p[n] : 1.f, min_p = a.min_p ? a.min_p[n] : 0.f;
    const int top_k = a.top_k ? a.top_k[n] : 0;
    const bool by_p = top_p < 1.f, by_k = top_k > 0 && top_k < V;
    u64 cut = ~0ull;   // the last place that is kept
    if (by_p || by_k) {
        for (int i = tid; i < V; i += kThreads) {
            const float y = value(x, i);
            if (y != y) continue;
            const int b = row.bin(y);
            atomicAdd(&sh.count[b], 1u);
            if (by_p) atomicAdd(&sh.mass[b], row.weight(y));
        }
        __syncthreads();
        int bin = -1;      // whose logits the list holds
        const auto cut_in = [&](int b, auto by_mass, u64 want, u64 &upto) {
            constexpr bool MASS = decltype(by_mass)::value;
            const bool few = sh.count[b] <= (uint32_t)kList;
            if (few && bin != b) {
                if (tid == 0) sh.listed = 0;
                __syncthreads();
                for (int i = tid; i < V; i += kThreads) {
                    const float y = value(x, i);
                    if (y == y && row.bin(y) == b) sh.list[atomicAdd(&sh.listed, 1)] = place_of<T>(y, i);
                }
                __syncthreads();
                bin = b;
            }
            if (few) {
                const int some = sh.listed;
                const auto each = [&](auto f) {
                    for (int i = tid; i < some; i += kThreads) {
                        const u64 p = sh.list[i];
                        f(p, value(x, (uint32_t)p));
                    }
                };
                return select<T, MASS>(sh, row, each, index_bits, want, upto);
            }
            const auto each = [&](auto f) {
                for (int i = tid; i < V; i += kThreads) {
                    const float y = value(x, i);
                    if (y == y && row.bin(y) == b) f(place_of<T>(y, i), y);
                }
            };
            return select<T, MASS>(sh, row, each, index_bits, want, upto);
        };
        // bins up to one: their weights, and the first at which counts or weights reach
        const auto reach = [&](const auto *of, u64 want, u64 &before) {
            if (tid < 64) {
                u64 sum;
                const int b = first_reaching(of, kBins, want, sum);
                if (tid == 0) {
                    sh.out[0] = b;
                    sh.out[1] = sum;
                }
            }
            __syncthreads();
            const int b = (int)sh.out[0];
            before = sh.out[1];
            __syncthreads();
            return b;
        };
        const auto mass_below = [&](int b) {
            u64 s = 0;
            for (int i = tid; i < b; i += kThreads) s += sh.mass[i];
            s = wave_sum(s);
            if (lane == 0) sh.sums[wave] = s;
            __syncthreads();
            s = 0;
            for (int w = 0; w < kWaves; ++w) s += sh.sums[w];
            __syncthreads();
            return s;
        };
        u64 total = 0, before;
        int last = kBins;
        if (by_k) {
            last = reach(sh.count, (u64)top_k, before);
            if (last < kBins) {
                u64 upto;
                cut = cut_in(last, std::false_type{}, (u64)top_k - before, upto);
                total = by_p ? mass_below(last) + upto : 0;
            }
        }
        if (by_p) {
            if (last == kBins) total = mass_below(kBins);
            const double part = (double)__builtin_fmaxf(top_p, 0.f) * (double)total;
            u64 want = (u64)part;
            if ((double)want < part) ++want;
            want = max(min(want, total), (u64)1);
            const int b = reach(sh.mass, want, before);
            u64 upto;
            cut = min(cut, cut_in(b, std::true_type{}, want - before, upto));
        }
    }

    // what is kept of the weights, by sixteenths of what is left of the row
    const double least = min_p > 0.f ? (double)__builtin_fminf(min_p, 1.f) * row.one : 0.0;
    const auto kept = [&](int i) -> u64 {
        const float y = value(x, i);
        if (y != y || place_of<T>(y, i) > cut) return 0;
        if (least > 0.0 && row.real(y) < least) return 0;
        return row.weight(y);
    };
    int lo = 0, hi = V;
    u64 want = 0, total = 0;
    for (bool firstly = true; firstly || hi - lo > 64; firstly = false) {
        const int each = (hi - lo + kWaves - 1) / kWaves, from = min(lo + wave * each, hi), to = min(from + each, hi);
        u64 s = 0;
        for (int i = from + lane; i < to; i += 64) s += kept(i);
        s = wave_sum(s);
        if (lane == 0) sh.sums[wave] = s;
        __syncthreads();
        if (firstly) {
            for (int w = 0; w < kWaves; ++w) total += sh.sums[w];
            if (!a.tokens) break;
            want = min((u64)((double)a.uniform[n] * (double)total), total - 1);   // the running sum is to pass this
        }
        int part = 0;
        for (; part < kWaves - 1 && sh.sums[part] <= want; ++part) want -= sh.sums[part];
        lo = min(lo + part * each, hi);
        hi = min(lo + each, hi);
        __syncthreads();
    }
    if (a.tokens && wave == 0) {
        u64 incl = lo + lane < hi ? kept(lo + lane) : 0;
#pragma unroll
        for (int m = 1; m < 64; m <<= 1) {
            const u64 y = __shfl_up(incl, m, 64);
            if (lane >= m) incl += y;
        }
        const u64 past = __ballot(incl > want);
        if (lane == 0) a.tokens[n] = lo + (past ? __builtin_ctzll(past) : 0);
    }
    if (probs) {
        const double f = 1.0 / (double)total;
        for (int i = tid; i < V; i += kThreads) {
            const float y = value(x, i);
            const bool in = y == y && place_of<T>(y, i) <= cut;
            const double w = in ? row.real(y) : 0.0;
            probs[i] = w < least ? 0.f : (float)(w * f);
        }
    }
}

}  // namespace

size_t sample_workspace_bytes(int, int, bool) { return 0; }

hipError_t launch_sample(const SampleArgs &a, void *, hipStream_t stream) {
    const int index_bits = 32 - __builtin_clz((unsigned)(a.vocab > 1 ? a.vocab - 1 : 1));
    const int bits = index_bits <= 16 ? 46 : 62 - index_bits;
    if (a.bf16) sample_kernel<bf16><<<a.rows, kThreads, 0, stream>>>(a, bits);
    else sample_kernel<float><<<a.rows, kThreads, 0, stream>>>(a, bits);
    return hipGetLastError();
}

}  // namespace kda
