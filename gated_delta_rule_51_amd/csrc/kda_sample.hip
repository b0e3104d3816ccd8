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
// Two launches.  The first cuts rows into parts, over the whole chip: each
// part's largest logit, and a histogram of counts and weights over bins of
// x / T, an eighth of a power of two wide and the same for all parts.  The
// second has one workgroup a row: the parts' histograms together say in which
// bin a cut lies, that bin's few logits are gathered and put in order, and the
// part that holds the token, known by its share of the weights, is gone through
// again.  A third writes the probabilities where they are asked for.
#include <algorithm>
#include <type_traits>

#include "kda_device.h"
#include "kda_internal.h"

namespace kda {
namespace {

constexpr int kThreads = 1024, kWaves = kThreads / 64, kPartThreads = 256;
constexpr int kBins = 256, kFine = 2048, kList = 4096, kFew = 256;
constexpr int kMostParts = 64;
// Up to this top_k the weights are not needed before the cut is known, so the
// first launch only counts.
constexpr int kCountOnly = 1024;
typedef unsigned long long u64;

__device__ __forceinline__ float value(const float *p, long i) { return p[i]; }
__device__ __forceinline__ float value(const bf16 *p, long i) { return bf16_to_f32(p[i].bits); }

// f(x, i) for the elements [lo, hi) of a row that starts anywhere, by THREADS
// threads, 16 bytes a load.
template <int THREADS, typename T, typename F> __device__ __forceinline__ void each_of(const T *x, int lo, int hi, F f) {
    constexpr int N = 16 / (int)sizeof(T);
    const int tid = threadIdx.x, head = min(hi - lo, (int)((0 - reinterpret_cast<uintptr_t>(x + lo)) % 16 / sizeof(T)));
    if (tid < head) f(value(x, lo + tid), lo + tid);
    const int from = lo + head, wide = (hi - from) / N;
    for (int v = tid; v < wide; v += THREADS) {
        const u32x4 w = *reinterpret_cast<const u32x4 *>(x + from + (long)v * N);
#pragma unroll
        for (int e = 0; e < N; ++e) {
            float y;
            if constexpr (N == 4) y = __uint_as_float(w[e]);
            else y = __uint_as_float(e & 1 ? w[e / 2] & 0xffff0000u : w[e / 2] << 16);
            f(y, from + v * N + e);
        }
    }
    const int tail = from + wide * N;
    if (tail + tid < hi) f(value(x, tail + tid), tail + tid);
}

// What a row's weights come from.
struct Row {
    float top;              // the largest logit
    float bins;             // bins of one unit of logits
    double rate;            // 64 log2(e) / T
    double one;             // 2^B
    const double *root;     // 2^(j / 64)

    // Rises with x, whatever x and the rate.
    __device__ __forceinline__ int bin(float x) const {
        constexpr float far = 536870912.f;
        return (int)__builtin_floorf(__builtin_fminf(__builtin_fmaxf(x * bins, -far), far));
    }
    // 2^B exp((x - top) / T): 2^(k / 64) from a table and e^r, |r| <= ln 2 / 128,
    // to r^5 (the rest is below 4e-17).
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
    // The same as a whole number.
    __device__ __forceinline__ u64 weight(float x) const {
        return (u64)__builtin_bit_cast(long long, real(x) + 4503599627370496.0) & 0xfffffffffffffull;   // 2^52: the fraction is the number
    }
};

__device__ __forceinline__ Row row_at(float top, float temperature, int bits, const double *root) {
    Row r;
    r.top = top;
    r.bins = __builtin_fmaxf(__builtin_fminf(8.f * kLog2e / temperature, 1e30f), 1e-37f);   // an infinity stays one
    r.rate = 64.0 * 1.4426950408889634074 / (double)temperature;
    r.one = (double)(1ull << bits);
    r.root = root;
    return r;
}

// 2^(j / 64)
__device__ __forceinline__ void fill_roots(double *root) {
    if (threadIdx.x < 64) root[threadIdx.x] = exp2((double)threadIdx.x / 64.0);
}

// What falls as x rises, 0 at the largest; both zeros are one.
__device__ __forceinline__ uint32_t key_of(float x) {
    const uint32_t b = x == 0.f ? 0 : __float_as_uint(x);
    return b >> 31 ? b : ~b & 0x7fffffffu;
}
__device__ __forceinline__ float of_key(uint32_t k) { return __uint_as_float(k >> 31 ? k : ~k & 0x7fffffffu); }

// Place in the order: smaller is earlier.  The key's bits lie at the top, 32 of
// them (16 for bf16), the index below.
template <typename T> __device__ __forceinline__ u64 place_of(float x, int i) {
    if constexpr (sizeof(T) == 2) return (u64)(key_of(x) >> 16) << 48 | (uint32_t)i;
    else return (u64)key_of(x) << 32 | (uint32_t)i;
}
// The last place whose logit is `k` or larger.
template <typename T> __device__ __forceinline__ u64 last_of_key(uint32_t k) {
    if constexpr (sizeof(T) == 2) return (u64)(k >> 31 ? k >> 16 : ((k + 1) >> 16) - 1) << 48 | 0xffffffffffffull;
    else return (u64)k << 32 | 0xffffffffull;
}

__device__ __forceinline__ u64 wave_sum(u64 x) {
#pragma unroll
    for (int m = 32; m >= 1; m >>= 1) x += __shfl_xor(x, m, 64);
    return x;
}
__device__ __forceinline__ u64 wave_running(u64 x) {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) {
        const u64 y = __shfl_up(x, m, 64);
        if (lane >= m) x += y;
    }
    return x;
}

// The largest of a workgroup's values and the first index that has it, in
// every thread.
template <int WAVES> __device__ __forceinline__ void block_top(float &top, int &at, float (&tops)[WAVES], int (&ats)[WAVES]) {
#pragma unroll
    for (int m = 32; m >= 1; m >>= 1) {
        const float y = __shfl_xor(top, m, 64);
        const int j = __shfl_xor(at, m, 64);
        if (y > top || (y == top && j < at)) {
            top = y;
            at = j;
        }
    }
    if ((threadIdx.x & 63) == 0) {
        tops[threadIdx.x >> 6] = top;
        ats[threadIdx.x >> 6] = at;
    }
    __syncthreads();
#pragma unroll
    for (int w = 0; w < WAVES; ++w)
        if (tops[w] > top || (tops[w] == top && ats[w] < at)) {
            top = tops[w];
            at = ats[w];
        }
}

// ---- first launch: the parts -------------------------------------------------

struct Part { float top; int at, bin, pad; };
enum Kind : int { kNothing, kLargest, kDrawn };
struct Chosen { u64 cut, total; float top; int at, kind, pad; };

struct Work {          // in the workspace
    int parts, length; // of a row; elements of a part
    Part *part;        // [rows, parts]
    Chosen *row;       // [rows]
    u64 *mass;         // [rows, parts, kBins]: weights against the part's largest, by bins below its first
    uint32_t *count;   // the same
};

struct Limits {
    float temperature, top_p, min_p;
    int top_k;
    bool by_k, by_p, by_m, counts;   // counts: the first launch only counts
};
__device__ __forceinline__ Limits limits_of(const SampleArgs &a, long n) {
    Limits y;
    y.temperature = a.temperature ? a.temperature[n] : 1.f;
    y.top_p = a.top_p ? a.top_p[n] : 1.f;
    y.min_p = a.min_p ? __builtin_fminf(a.min_p[n], 1.f) : 0.f;
    y.top_k = a.top_k ? a.top_k[n] : 0;
    y.by_k = y.top_k > 0 && y.top_k < a.vocab;
    y.by_p = y.top_p < 1.f;
    y.by_m = y.min_p > 0.f;
    y.counts = y.by_k && y.top_k <= kCountOnly;
    return y;
}

template <typename T> __global__ __launch_bounds__(kPartThreads) void parts_kernel(const SampleArgs a, const Work w, int bits) {
    __shared__ uint32_t count[kBins];
    __shared__ u64 mass[kBins];
    __shared__ double root[64];
    __shared__ float tops[kPartThreads / 64];
    __shared__ int ats[kPartThreads / 64];
    const int tid = threadIdx.x, lo = (blockIdx.x % w.parts) * w.length, hi = min(lo + w.length, a.vocab);
    const long n = blockIdx.x / w.parts;
    const T *x = static_cast<const T *>(a.logits) + n * a.stride;
    const Limits lim = limits_of(a, n);
    count[tid] = 0;
    mass[tid] = 0;
    fill_roots(root);
    float top = -__builtin_inff();
    int at = INT32_MAX;
    each_of<kPartThreads>(x, lo, hi, [&](float y, int i) {
        if (y > top || (y == top && i < at)) {
            top = y;
            at = i;
        }
    });
    block_top(top, at, tops, ats);
    const bool some = top > -__builtin_inff() && lim.temperature > 0.f;
    const Row row = row_at(top, lim.temperature, bits, root);
    const int first = some ? row.bin(top) : 0;
    if (tid == 0) w.part[blockIdx.x] = Part{top, at, first, 0};
    if (!some) return;
    each_of<kPartThreads>(x, lo, hi, [&](float y, int) {
        if (y != y) return;
        const int b = (int)min((uint32_t)(first - row.bin(y)), (uint32_t)kBins - 1);
        atomicAdd(&count[b], 1u);
        if (!lim.counts) atomicAdd(&mass[b], row.weight(y));
    });
    __syncthreads();
    w.count[(long)blockIdx.x * kBins + tid] = count[tid];
    if (!lim.counts) w.mass[(long)blockIdx.x * kBins + tid] = mass[tid];
}

// ---- second launch: the cut and the token --------------------------------------

struct Shared {
    uint32_t count[kFine];
    u64 mass[kFine];
    u64 list[kList];
    u64 sorted[kFew], sorted_mass[kFew];
    uint32_t rank[kFew];
    double root[64];
    uint32_t digit[256];
    u64 digit_mass[256];
    u64 sums[kWaves], part_mass[kMostParts];
    double factor[kMostParts];
    int shift[kMostParts];
    u64 out[4];
    float tops[kWaves];
    int ats[kWaves];
    int listed;
};

// The first of n numbers (n a multiple of 64) with which their running sum is
// at least `want`, by one wave; `before`: the sum up to it.  n where there is
// none.
template <typename N> __device__ __forceinline__ int first_reaching(const N *at, int n, u64 want, u64 &before) {
    const int lane = threadIdx.x & 63;
    u64 sum = 0;
    for (int i = 0; i < n; i += 64) {
        const u64 own = at[i + lane], incl = wave_running(own) + sum;
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
// The same for the whole workgroup.
template <typename N> __device__ __forceinline__ int block_reaching(Shared &sh, const N *at, int n, u64 want, u64 &before) {
    if (threadIdx.x < 64) {
        u64 sum;
        const int b = first_reaching(at, n, want, sum);
        if (threadIdx.x == 0) {
            sh.out[0] = b;
            sh.out[1] = sum;
        }
    }
    __syncthreads();
    const int b = (int)sh.out[0];
    before = sh.out[1];
    __syncthreads();
    return b;
}
__device__ __forceinline__ u64 block_sum(Shared &sh, u64 x) {
    x = wave_sum(x);
    if ((threadIdx.x & 63) == 0) sh.sums[threadIdx.x >> 6] = x;
    __syncthreads();
    x = 0;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) x += sh.sums[w];
    __syncthreads();
    return x;
}

// Among the places each() goes over, the first at which the running count (or
// sum of weights, BY_MASS) is at least `want`, digit by digit; `upto`: the sum of
// weights up to it and its own.
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
            if constexpr (BY_MASS) d = min(first_reaching(sh.digit_mass, 256, want, before), 255);
            else d = min(first_reaching(sh.digit, 256, want, before), 255);
            u64 less = 0;   // weights of the digits below
            for (int i = tid; i < d; i += 64) less += sh.digit_mass[i];
            less = wave_sum(less);
            if (tid == 0) {
                sh.out[0] = d;
                sh.out[1] = want - min(before, want);
                sh.out[2] = less;
                sh.out[3] = sh.digit_mass[d];
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

// Up to kFew places of sh.list put in order, with their weights.
template <typename T> __device__ __forceinline__ void sort_few(Shared &sh, const Row &row, const T *x, int n) {
    const int tid = threadIdx.x;
    if (tid < kFew) sh.rank[tid] = 0;
    __syncthreads();
    // every place against the others, a quarter of them a thread
    const int mine = tid & (kFew - 1), from = tid / kFew * (kFew / 4), to = min(from + kFew / 4, n);
    const u64 p = sh.list[mine];
    if (mine < n) {
        uint32_t r = 0;
        for (int i = from; i < to; ++i) r += sh.list[i] < p;
        if (r) atomicAdd(&sh.rank[mine], r);
    }
    __syncthreads();
    if (tid < n) {
        sh.sorted[sh.rank[tid]] = p;
        sh.sorted_mass[sh.rank[tid]] = row.weight(value(x, (uint32_t)p));
    }
    __syncthreads();
}

// Gathers the places of a row's logits that in() picks into sh.list; as many as
// the caller has counted.
template <typename T, typename In> __device__ __forceinline__ void gather(Shared &sh, const T *x, int V, const In &in) {
    if (threadIdx.x == 0) sh.listed = 0;
    __syncthreads();
    each_of<kThreads>(x, 0, V, [&](float y, int i) {
        if (y == y && in(y)) {
            const int at = atomicAdd(&sh.listed, 1);
            if (at < kList) sh.list[at] = place_of<T>(y, i);
        }
    });
    __syncthreads();
}

// The cut of a row whatever its logits, from passes over all of it: for rows
// with more logits in the cut's bin than the list holds (thousands of equal
// ones, or a cut far down).
template <typename T> __device__ u64 cut_of_whole_row(Shared &sh, const Row &row, const Limits &lim, const T *x, int V, int index_bits) {
    const int tid = threadIdx.x;
    // bins of (top - x) / T, 64 a unit
    const float rate = 64.f / lim.temperature;
    const auto bin = [&](float y) {
        const float z = (row.top - y) * rate;
        return z < (float)(kFine - 1) ? (int)z : z >= 0.f ? kFine - 1 : 0;
    };
    for (int i = tid; i < kFine; i += kThreads) {
        sh.count[i] = 0;
        sh.mass[i] = 0;
    }
    __syncthreads();
    for (int i = tid; i < V; i += kThreads) {
        const float y = value(x, i);
        if (y != y) continue;
        const int b = bin(y);
        atomicAdd(&sh.count[b], 1u);
        atomicAdd(&sh.mass[b], row.weight(y));
    }
    __syncthreads();
    const auto cut_in = [&](int b, auto by_mass, u64 want, u64 &upto) {
        const auto each = [&](auto f) {
            for (int i = tid; i < V; i += kThreads) {
                const float y = value(x, i);
                if (y == y && bin(y) == b) f(place_of<T>(y, i), y);
            }
        };
        return select<T, decltype(by_mass)::value>(sh, row, each, index_bits, want, upto);
    };
    u64 cut = ~0ull, before, upto = 0;
    int last = kFine;
    if (lim.by_k) {
        last = block_reaching(sh, sh.count, kFine, (u64)lim.top_k, before);
        if (last < kFine) cut = cut_in(last, std::false_type{}, (u64)lim.top_k - before, upto);
    }
    if (lim.by_p) {
        u64 s = 0;
        for (int i = tid; i < last; i += kThreads) s += sh.mass[i];
        const u64 total = block_sum(sh, s) + upto;
        const double part = (double)__builtin_fmaxf(lim.top_p, 0.f) * (double)total;
        const u64 want = max(min((u64)__builtin_ceil(part), total), (u64)1);
        const int b = block_reaching(sh, sh.mass, kFine, want, before);
        cut = min(cut, cut_in(min(b, kFine - 1), std::true_type{}, want - before, upto));
    }
    return cut;
}

template <typename T> __global__ __launch_bounds__(kThreads) void choose_kernel(const SampleArgs a, const Work w, int bits) {
    __shared__ Shared sh;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, V = a.vocab;
    const long n = blockIdx.x;
    const T *x = static_cast<const T *>(a.logits) + n * a.stride;
    const Limits lim = limits_of(a, n);
    const Part *parts = w.part + n * w.parts;

    float top = -__builtin_inff();
    int at = INT32_MAX;
    for (int p = 0; p < w.parts; ++p)
        if (parts[p].top > top) {
            top = parts[p].top;
            at = parts[p].at;
        }
    if (!(top > -__builtin_inff()) || !(lim.temperature > 0.f)) {   // no logit at all, or the largest
        if (tid == 0) {
            const bool none = !(top > -__builtin_inff());
            if (a.tokens) a.tokens[n] = none ? -1 : at;
            w.row[n] = Chosen{0, 0, top, at, none ? kNothing : kLargest, 0};
        }
        return;
    }
    fill_roots(sh.root);
    const Row row = row_at(top, lim.temperature, bits, sh.root);
    const int first = row.bin(top), index_bits = 32 - __builtin_clz(max(V - 1, 1));
    const auto bin = [&](float y) { return (int)min((uint32_t)(first - row.bin(y)), (uint32_t)kBins - 1); };
    __syncthreads();
    // the parts' bins and weights against the row's largest
    if (tid < w.parts) {
        sh.shift[tid] = min(first - parts[tid].bin, kBins - 1);
        sh.factor[tid] = parts[tid].top > -__builtin_inff() ? row.real(parts[tid].top) / row.one : -1.0;   // -1: nothing there
    }
    if (tid < kBins) {
        sh.count[tid] = 0;
        sh.mass[tid] = 0;
    }
    __syncthreads();
    if (lim.by_k || lim.by_p) {
        const int j = tid & (kBins - 1);
        for (int p = tid / kBins; p < w.parts; p += kThreads / kBins) {
            if (sh.factor[p] < 0.0) continue;
            const long from = (n * w.parts + p) * kBins + j;
            const uint32_t y = w.count[from];
            const u64 z = lim.counts ? 0 : (u64)__builtin_rint((double)w.mass[from] * sh.factor[p]);
            const int to = min(j + sh.shift[p], kBins - 1);
            atomicAdd(&sh.count[to], y);
            if (!lim.counts) atomicAdd(&sh.mass[to], z);
        }
        __syncthreads();
    }

    u64 cut = ~0ull;                 // the last place that is kept
    if (lim.by_m) {                  // the smallest number whose weight is not below the limit
        if (wave == 0) {
            const double least = (double)lim.min_p * row.one;
            uint32_t lo = key_of(top), hi = 0xff800000u;   // holds; does not (minus infinity weighs nothing)
            while (hi - lo > 1) {
                const uint32_t step = (hi - lo + 63) / 64;
                const uint32_t k = (uint32_t)min((u64)lo + (u64)step * lane, (u64)hi);
                const u64 holds = __ballot(k < hi && (k == lo || row.real(of_key(k)) >= least));
                const int last = 63 - __builtin_clzll(holds);
                hi = (uint32_t)min((u64)lo + (u64)step * (last + 1), (u64)hi);
                lo += step * last;
            }
            if (lane == 0) sh.out[0] = last_of_key<T>(lo);
        }
        __syncthreads();
        cut = sh.out[0];
        __syncthreads();
    }

    bool whole = false;              // the list cannot hold a cut's bin
    u64 total = 0;                   // of the weights kept
    if (lim.counts) {
        // few are kept: all logits up to the bin of the k-th
        u64 before;
        const int b = min(block_reaching(sh, sh.count, kBins, (u64)lim.top_k, before), kBins - 1);
        u64 c = tid <= b ? sh.count[tid] : 0;
        const int some = (int)min(block_sum(sh, c), (u64)kList + 1);
        whole = some > kList;
        if (!whole) {
            gather(sh, x, V, [&](float y) { return bin(y) <= b; });
            if (some <= kFew) {
                sort_few(sh, row, x, some);
                int keep = min(some, lim.top_k);
                if (wave == 0) {
                    // running sums, four a lane
                    u64 y[4], s = 0;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        y[i] = 4 * lane + i < keep ? sh.sorted_mass[4 * lane + i] : 0;
                        s += y[i];
                    }
                    const u64 incl = wave_running(s), all = __shfl(incl, 63, 64);
                    u64 want = all;
                    if (lim.by_p) want = max(min((u64)__builtin_ceil((double)__builtin_fmaxf(lim.top_p, 0.f) * (double)all), all), (u64)1);
                    u64 run = incl - s;
                    int mine = 0;      // of this lane's four, those kept
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int k = 4 * lane + i;
                        if (k < keep && (!lim.by_p || run < want) && sh.sorted[k] <= cut) ++mine;
                        run += y[i];
                    }
#pragma unroll
                    for (int m = 32; m >= 1; m >>= 1) mine += __shfl_xor(mine, m, 64);
                    u64 kept = 0;
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (4 * lane + i < mine) kept += y[i];
                    kept = wave_sum(kept);
                    if (lane == 0) {
                        sh.out[0] = mine;
                        sh.out[1] = kept;
                    }
                }
                __syncthreads();
                keep = (int)sh.out[0];
                total = sh.out[1];
                cut = sh.sorted[keep - 1];
                if (a.tokens && tid < keep) {
                    // the running sum by index of every logit kept
                    const u64 want = min((u64)((double)a.uniform[n] * (double)total), total - 1);
                    const uint32_t i = (uint32_t)sh.sorted[tid];
                    const u64 own = sh.sorted_mass[tid];
                    u64 below = 0;
                    for (int j = 0; j < keep; ++j)
                        if ((uint32_t)sh.sorted[j] < i) below += sh.sorted_mass[j];
                    if (below <= want && below + own > want) a.tokens[n] = (int)i;
                }
                if (tid == 0) w.row[n] = Chosen{cut, total, top, at, kDrawn, 0};
                return;
            }
            const auto each = [&](auto f) {
                for (int i = tid; i < some; i += kThreads) {
                    const u64 p = sh.list[i];
                    f(p, value(x, (uint32_t)p));
                }
            };
            u64 all;
            if (some > lim.top_k) {
                cut = min(cut, select<T, false>(sh, row, each, index_bits, (u64)lim.top_k, all));
            } else {
                u64 s = 0;
                each([&](u64, float y) { s += row.weight(y); });
                all = block_sum(sh, s);
            }
            if (lim.by_p) {
                const u64 want = max(min((u64)__builtin_ceil((double)__builtin_fmaxf(lim.top_p, 0.f) * (double)all), all), (u64)1);
                u64 upto;
                cut = min(cut, select<T, true>(sh, row, each, index_bits, want, upto));
            }
            // drawn by index: the place is the index alone
            u64 s = 0;
            each([&](u64 p, float y) { s += p <= cut ? row.weight(y) : 0; });
            total = block_sum(sh, s);
            if (a.tokens) {
                const auto by_index = [&](auto f) {
                    each([&](u64 p, float y) {
                        if (p <= cut) f((u64)(uint32_t)p, y);
                    });
                };
                const u64 want = min((u64)((double)a.uniform[n] * (double)total), total - 1) + 1;
                u64 upto;
                const u64 i = select<float, true>(sh, row, by_index, index_bits, want, upto);
                if (tid == 0) a.tokens[n] = (int)i;
            }
            if (tid == 0) w.row[n] = Chosen{cut, total, top, at, kDrawn, 0};
            return;
        }
    }
    int edge = kBins;                // the bin that the cut goes through: those before it are kept whole
    int listed = -1;                 // the bin whose logits the list holds, in order where they are few
    if (!lim.counts) {
        const auto list = [&](int b) {
            if (listed == b) return;
            gather(sh, x, V, [&](float y) { return bin(y) == b; });
            if (sh.listed <= kFew) sort_few(sh, row, x, sh.listed);
            listed = b;
        };
        const auto cut_in = [&](int b, auto by_mass, u64 want, u64 &upto) -> u64 {
            constexpr bool MASS = decltype(by_mass)::value;
            list(b);
            const int some = sh.listed;
            upto = 0;
            if (some == 0) return ~0ull;   // sums that differ in the last place ended up behind the last logit
            if (some > kFew) {
                const auto each = [&](auto f) {
                    for (int i = tid; i < some; i += kThreads) {
                        const u64 p = sh.list[i];
                        f(p, value(x, (uint32_t)p));
                    }
                };
                return select<T, MASS>(sh, row, each, index_bits, want, upto);
            }
            if (wave == 0) {
                u64 y[4], s = 0;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    y[i] = 4 * lane + i < some ? sh.sorted_mass[4 * lane + i] : 0;
                    s += y[i];
                }
                u64 run = wave_running(s) - s;
                int mine = 0;      // of this lane's four, those kept
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int k = 4 * lane + i;
                    if (k < some && (MASS ? run < want : (u64)k < want)) ++mine;
                    run += y[i];
                }
#pragma unroll
                for (int m = 32; m >= 1; m >>= 1) mine += __shfl_xor(mine, m, 64);
                u64 kept = 0;
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (4 * lane + i < mine) kept += y[i];
                kept = wave_sum(kept);
                if (lane == 0) {
                    sh.out[0] = sh.sorted[max(mine - 1, 0)];
                    sh.out[1] = kept;
                }
            }
            __syncthreads();
            const u64 c = sh.out[0];
            upto = sh.out[1];
            __syncthreads();
            return c;
        };
        u64 before, upto = 0;
        int last = kBins;
        if (lim.by_k) {
            last = block_reaching(sh, sh.count, kBins, (u64)lim.top_k, before);
            if (last < kBins) {
                whole = sh.count[last] > (uint32_t)kList;
                if (!whole) {
                    cut = min(cut, cut_in(last, std::false_type{}, (u64)lim.top_k - before, upto));
                    edge = last;
                }
            }
        }
        if (lim.by_p && !whole) {
            const u64 all = block_sum(sh, tid < last && tid < kBins ? sh.mass[tid] : 0) + upto;
            const u64 want = max(min((u64)__builtin_ceil((double)__builtin_fmaxf(lim.top_p, 0.f) * (double)all), all), (u64)1);
            const int b = min(block_reaching(sh, sh.mass, kBins, want, before), kBins - 1);
            whole = sh.count[b] > (uint32_t)kList;
            if (!whole) {
                cut = min(cut, cut_in(b, std::true_type{}, want - min(before, want), upto));
                edge = min(edge, b);
            }
        }
        if (lim.by_m && !whole) {    // the bin of the limit's own number; the list may not hold it
            const uint32_t k = (uint32_t)(cut >> 32);
            const float y = of_key(sizeof(T) == 2 ? (k >> 31 ? k & 0xffff0000u : k | 0xffffu) : k);
            if (bin(y) < edge) {
                edge = bin(y);
                u64 c = 0;
                if (!(lim.by_k || lim.by_p)) {   // its bins were not brought together
                    const int p = tid;
                    if (p < w.parts && sh.factor[p] >= 0.0) {
                        const int j = edge - sh.shift[p];
                        if (edge < kBins - 1) c = j >= 0 ? w.count[(n * w.parts + p) * kBins + j] : 0;
                        else
                            for (int i = max(j, 0); i < kBins; ++i) c += w.count[(n * w.parts + p) * kBins + i];
                    }
                    c = block_sum(sh, c);
                } else {
                    c = sh.count[edge];
                }
                whole = c > (u64)kList;
            }
        }
        if (!whole && edge < kBins) list(edge);
    }
    if (whole) {
        __syncthreads();
        const u64 least = cut;
        cut = min(lim.by_m ? least : ~0ull, cut_of_whole_row(sh, row, lim, x, V, index_bits));
    }

    const auto kept = [&](int i) -> u64 {
        const float y = value(x, i);
        return y == y && place_of<T>(y, i) <= cut ? row.weight(y) : 0;
    };
    int lo = 0, hi = V;
    u64 want = 0;
    if (!whole) {
        // what every part keeps: its bins before the cut's, and its share of the list
        if (listed >= 0) {
            if (tid < kMostParts) sh.part_mass[tid] = 0;
            __syncthreads();
            const int some = sh.listed;
            for (int i = tid; i < some; i += kThreads) {
                const u64 p = sh.list[i];
                if (p <= cut) {
                    const float y = value(x, (uint32_t)p);
                    if (bin(y) == edge) atomicAdd(&sh.part_mass[(uint32_t)p / (uint32_t)w.length], row.weight(y));
                }
            }
            __syncthreads();
        }
        for (int p = wave; p < w.parts; p += kWaves) {
            if (sh.factor[p] < 0.0) {
                if (lane == 0) sh.part_mass[p] = 0;
                continue;
            }
            u64 s = 0;
            for (int j = lane; j < kBins; j += 64)
                if (edge == kBins || min(j + sh.shift[p], kBins - 1) < edge) s += w.mass[(n * w.parts + p) * kBins + j];
            s = wave_sum(s);
            if (lane == 0) sh.part_mass[p] = (u64)__builtin_rint((double)s * sh.factor[p]) + (listed >= 0 ? sh.part_mass[p] : 0);
        }
        if (tid < kMostParts && tid >= w.parts) sh.part_mass[tid] = 0;
        __syncthreads();
        if (wave == 0) {
            const u64 own = sh.part_mass[lane], incl = wave_running(own), all = __shfl(incl, 63, 64);
            u64 to = 0;
            if (a.tokens) to = min((u64)((double)a.uniform[n] * (double)all), all - 1);
            const u64 past = __ballot(incl > to);
            const int p = past ? __builtin_ctzll(past) : 0;
            const u64 rest = to - __shfl(incl - own, p, 64);
            if (lane == 0) {
                sh.out[0] = p;
                sh.out[1] = rest;
                sh.out[2] = all;
            }
        }
        __syncthreads();
        lo = (int)sh.out[0] * w.length;
        hi = min(lo + w.length, V);
        want = sh.out[1];
        total = sh.out[2];
        __syncthreads();
    }
    if (tid == 0 && !whole) w.row[n] = Chosen{cut, total, top, at, kDrawn, 0};
    if (!whole && !a.tokens) return;
    // by sixteenths of what is left of the row
    for (bool firstly = whole; firstly || hi - lo > 64; firstly = false) {
        const int each = (hi - lo + kWaves - 1) / kWaves, from = min(lo + wave * each, hi), to = min(from + each, hi);
        u64 s = 0;
        for (int i = from + lane; i < to; i += 64) s += kept(i);
        s = wave_sum(s);
        if (lane == 0) sh.sums[wave] = s;
        __syncthreads();
        if (firstly) {
            total = 0;
            for (int i = 0; i < kWaves; ++i) total += sh.sums[i];
            if (tid == 0) w.row[n] = Chosen{cut, total, top, at, kDrawn, 0};
            if (!a.tokens) return;
            want = min((u64)((double)a.uniform[n] * (double)total), total - 1);   // the running sum is to pass this
        }
        int part = 0;
        for (; part < kWaves - 1 && sh.sums[part] <= want; ++part) want -= sh.sums[part];
        lo = min(lo + part * each, hi);
        hi = min(lo + each, hi);
        __syncthreads();
    }
    if (wave == 0) {
        const u64 own = lo + lane < hi ? kept(lo + lane) : 0, incl = wave_running(own);
        // the sums of parts and of their logits may differ in the last place: then the last one that weighs
        const u64 past = __ballot(incl > want), some = __ballot(own > 0);
        if (lane == 0) a.tokens[n] = lo + (past ? __builtin_ctzll(past) : some ? 63 - __builtin_clzll(some) : 0);
    }
}

// ---- third launch: the probabilities ---------------------------------------------

template <typename T> __global__ __launch_bounds__(kPartThreads) void probs_kernel(const SampleArgs a, const Work w, int bits) {
    __shared__ double root[64];
    const int lo = (blockIdx.x % w.parts) * w.length, hi = min(lo + w.length, a.vocab);
    const long n = blockIdx.x / w.parts;
    const T *x = static_cast<const T *>(a.logits) + n * a.stride;
    float *probs = a.probs + n * a.vocab;
    const Chosen c = w.row[n];
    if (c.kind != kDrawn) {
        for (int i = lo + threadIdx.x; i < hi; i += kPartThreads) probs[i] = c.kind == kLargest && i == c.at ? 1.f : 0.f;
        return;
    }
    fill_roots(root);
    __syncthreads();
    const Row row = row_at(c.top, a.temperature ? a.temperature[n] : 1.f, bits, root);
    const double f = 1.0 / (double)c.total;
    for (int i = lo + threadIdx.x; i < hi; i += kPartThreads) {
        const float y = value(x, i);
        probs[i] = y == y && place_of<T>(y, i) <= c.cut ? (float)(row.real(y) * f) : 0.f;
    }
}

size_t round_up(size_t n) { return (n + 255) / 256 * 256; }

// Parts of a row: enough workgroups for the chip, of 2048 logits or more.
void lay_out(Work &w, int rows, int vocab, void *workspace, size_t &bytes) {
    const long most = std::min<long>(kMostParts, (vocab + 2047) / 2048);
    w.parts = (int)std::max<long>(1, std::min<long>(most, (1024 + rows - 1) / rows));
    w.length = ((vocab + w.parts - 1) / w.parts + 7) / 8 * 8;
    w.parts = (vocab + w.length - 1) / w.length;
    const size_t cells = (size_t)rows * w.parts;
    char *at = static_cast<char *>(workspace);
    w.row = reinterpret_cast<Chosen *>(at);
    at += round_up(rows * sizeof(Chosen));
    w.part = reinterpret_cast<Part *>(at);
    at += round_up(cells * sizeof(Part));
    w.mass = reinterpret_cast<u64 *>(at);
    at += cells * kBins * sizeof(u64);
    w.count = reinterpret_cast<uint32_t *>(at);
    at += cells * kBins * sizeof(uint32_t);
    bytes = at - static_cast<char *>(workspace);
}

template <typename T> hipError_t launch(const SampleArgs &a, const Work &w, int bits, hipStream_t stream) {
    parts_kernel<T><<<(unsigned)(a.rows * w.parts), kPartThreads, 0, stream>>>(a, w, bits);
    choose_kernel<T><<<a.rows, kThreads, 0, stream>>>(a, w, bits);
    if (a.probs) probs_kernel<T><<<(unsigned)(a.rows * w.parts), kPartThreads, 0, stream>>>(a, w, bits);
    return hipGetLastError();
}

}  // namespace

size_t sample_workspace_bytes(int rows, int vocab) {
    Work w{};
    size_t bytes = 0;
    lay_out(w, rows, vocab, nullptr, bytes);
    return bytes;
}

hipError_t launch_sample(const SampleArgs &a, void *workspace, hipStream_t stream) {
    const int index_bits = 32 - __builtin_clz((unsigned)(a.vocab > 1 ? a.vocab - 1 : 1));
    const int bits = index_bits <= 16 ? 46 : 62 - index_bits;
    Work w{};
    size_t bytes;
    lay_out(w, a.rows, a.vocab, workspace, bytes);
    return a.bf16 ? launch<bf16>(a, w, bits, stream) : launch<float>(a, w, bits, stream);
}

}  // namespace kda
