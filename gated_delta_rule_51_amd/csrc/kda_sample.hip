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
// Neither does minus infinity, which masked rows are full of: it is left out from the
// start (one row of 131,072 with 20 tokens allowed, top_k 50: 24 us, unmasked 28).
//
// Two launches.  The first cuts rows into parts, over the whole chip: each
// part's largest logit, and a histogram of counts and weights over bins of
// x / T, an eighth of a power of two wide and the same for all parts.  The
// second has one workgroup a row: the parts' histograms together say in which
// bin a cut lies, that bin's few logits are gathered and put in order, and the
// part that holds the token, known by its share of the weights, is gone through
// again.  A third writes the probabilities where they are asked for.
//
// The first launch is bound by the vector units, that is by the weights in 64 bits
// (256 rows of 65,536 in bf16 21.5 us; with counts alone, 128 rows of 50,001 in fp32,
// 12), the second by the latency of one workgroup a row (one row of 131,072 27 us,
// 256 rows 33), the third by HBM (128 x 50,001 13.5 us, 3.8 TB/s).
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
// threads, 16 bytes a load, AHEAD loads at a time: a row's few workgroups wait
// for memory otherwise.
template <int THREADS, int AHEAD, typename T, typename F> __device__ __forceinline__ void each_of(const T *x, int lo, int hi, F f) {
    constexpr int N = 16 / (int)sizeof(T);
    const int tid = threadIdx.x, head = min(hi - lo, (int)((0 - reinterpret_cast<uintptr_t>(x + lo)) % 16 / sizeof(T)));
    if (tid < head) f(value(x, lo + tid), lo + tid);
    const int from = lo + head, wide = (hi - from) / N;
    for (int v = tid; v < wide; v += AHEAD * THREADS) {
        u32x4 w[AHEAD];
#pragma unroll
        for (int k = 0; k < AHEAD; ++k) w[k] = *reinterpret_cast<const u32x4 *>(x + from + (long)min(v + k * THREADS, wide - 1) * N);
#pragma unroll
        for (int k = 0; k < AHEAD; ++k) {
            if (v + k * THREADS >= wide) break;
#pragma unroll
            for (int e = 0; e < N; ++e) {
                float y;
                if constexpr (N == 4) y = __uint_as_float(w[k][e]);
                else y = __uint_as_float(e & 1 ? w[k][e / 2] & 0xffff0000u : w[k][e / 2] << 16);
                f(y, from + (v + k * THREADS) * N + e);
            }
        }
    }
    const int tail = from + wide * N;
    if (tail + tid < hi) f(value(x, tail + tid), tail + tid);
}

// What a row's weights come from.
struct Row {
    float top;              // the largest logit
    float bins;             // bins of one unit of logits
    double rate, shift;     // 64 log2(e) / T; top times that
    double one;             // 2^B
    const double *root;     // 2^(B + j / 64)

    // Rises with x, whatever x and the rate.
    __device__ __forceinline__ int bin(float x) const {
        constexpr float far = 536870912.f;
        return (int)__builtin_floorf(__builtin_fminf(__builtin_fmaxf(x * bins, -far), far));
    }
    // 2^B exp((x - top) / T) = 2^(B + z / 64): 2^(B + k / 64) for k = z rounded from a
    // table and its exponent, and 2^(r / 64), |r| <= 1/2, as its series to r^5 (the
    // rest is below 4e-17).  One fused operation forms z, so that top * rate, which
    // is rounded, is a factor that all weights but the largest have in common, off
    // by 2^-53 |top / T|.  What is below 2^-1000 counts as that.
    __device__ __forceinline__ double real(float x) const {
        const double z = __builtin_fmax(__builtin_fma((double)x, rate, -shift), -64000.0);
        const double k = __builtin_rint(z), r = z - k;
        double y = __builtin_fma(r, 0x1.5d87fe78a6730p-40, 0x1.3b2ab6fba4e77p-31);
        y = __builtin_fma(r, y, 0x1.c6b08d704a0bfp-23);
        y = __builtin_fma(r, y, 0x1.ebfbdff82c58ep-15);
        y = __builtin_fma(r, y, 0x1.62e42fefa39efp-7);
        y = __builtin_fma(r, y, 1.0);
        const int n = (int)k;
        const u64 bits = __builtin_bit_cast(u64, y * root[n & 63]) + ((u64)(uint32_t)(n >> 6) << 52);
        return x == top ? one : __builtin_bit_cast(double, bits);
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
    r.shift = (double)top * r.rate;
    r.one = (double)(1ull << bits);
    r.root = root;
    return r;
}

// 2^(j / 64), correctly rounded.
__constant__ const double kRoots[64] = {
    0x1.0000000000000p+0, 0x1.02c9a3e778061p+0, 0x1.059b0d3158574p+0, 0x1.0874518759bc8p+0,
    0x1.0b5586cf9890fp+0, 0x1.0e3ec32d3d1a2p+0, 0x1.11301d0125b51p+0, 0x1.1429aaea92de0p+0,
    0x1.172b83c7d517bp+0, 0x1.1a35beb6fcb75p+0, 0x1.1d4873168b9aap+0, 0x1.2063b88628cd6p+0,
    0x1.2387a6e756238p+0, 0x1.26b4565e27cddp+0, 0x1.29e9df51fdee1p+0, 0x1.2d285a6e4030bp+0,
    0x1.306fe0a31b715p+0, 0x1.33c08b26416ffp+0, 0x1.371a7373aa9cbp+0, 0x1.3a7db34e59ff7p+0,
    0x1.3dea64c123422p+0, 0x1.4160a21f72e2ap+0, 0x1.44e086061892dp+0, 0x1.486a2b5c13cd0p+0,
    0x1.4bfdad5362a27p+0, 0x1.4f9b2769d2ca7p+0, 0x1.5342b569d4f82p+0, 0x1.56f4736b527dap+0,
    0x1.5ab07dd485429p+0, 0x1.5e76f15ad2148p+0, 0x1.6247eb03a5585p+0, 0x1.6623882552225p+0,
    0x1.6a09e667f3bcdp+0, 0x1.6dfb23c651a2fp+0, 0x1.71f75e8ec5f74p+0, 0x1.75feb564267c9p+0,
    0x1.7a11473eb0187p+0, 0x1.7e2f336cf4e62p+0, 0x1.82589994cce13p+0, 0x1.868d99b4492edp+0,
    0x1.8ace5422aa0dbp+0, 0x1.8f1ae99157736p+0, 0x1.93737b0cdc5e5p+0, 0x1.97d829fde4e50p+0,
    0x1.9c49182a3f090p+0, 0x1.a0c667b5de565p+0, 0x1.a5503b23e255dp+0, 0x1.a9e6b5579fdbfp+0,
    0x1.ae89f995ad3adp+0, 0x1.b33a2b84f15fbp+0, 0x1.b7f76f2fb5e47p+0, 0x1.bcc1e904bc1d2p+0,
    0x1.c199bdd85529cp+0, 0x1.c67f12e57d14bp+0, 0x1.cb720dcef9069p+0, 0x1.d072d4a07897cp+0,
    0x1.d5818dcfba487p+0, 0x1.da9e603db3285p+0, 0x1.dfc97337b9b5fp+0, 0x1.e502ee78b3ff6p+0,
    0x1.ea4afa2a490dap+0, 0x1.efa1bee615a27p+0, 0x1.f50765b6e4540p+0, 0x1.fa7c1819e90d8p+0};
__device__ __forceinline__ void fill_roots(double *root, int bits) {
    if (threadIdx.x < 64) root[threadIdx.x] = kRoots[threadIdx.x] * (double)(1ull << bits);
}

// NaN is no logit, and minus infinity weighs nothing wherever a limit cuts: neither is
// counted or listed.  Whoever counts and whoever lists have to leave out the same.
__device__ __forceinline__ bool counted(float x) { return x > -__builtin_inff(); }

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
// A place's key, in its own 32 or 16 bits, and its logit.
template <typename T> __device__ __forceinline__ uint32_t place_key(u64 p) { return (uint32_t)(p >> (sizeof(T) == 2 ? 48 : 32)); }
template <typename T> __device__ __forceinline__ uint32_t cut_key(uint32_t key) { return sizeof(T) == 2 ? key >> 16 : key; }
template <typename T> __device__ __forceinline__ float place_value(u64 p) {
    const uint32_t k = place_key<T>(p);
    return of_key(sizeof(T) == 4 ? k : k >> 15 ? k << 16 : k << 16 | 0xffffu);
}
// The last place whose logit is `k` or larger.
template <typename T> __device__ __forceinline__ u64 last_of_key(uint32_t k) {
    if constexpr (sizeof(T) == 2) return (u64)(k >> 31 ? k >> 16 : ((k + 1) >> 16) - 1) << 48 | 0xffffffffffffull;
    else return (u64)k << 32 | 0xffffffffull;
}

// Sums over the wave's lanes up to each, and over all, without a trip through
// LDS.
template <int CTRL, int ROWS> __device__ __forceinline__ u64 dpp_plus(u64 x) {
    const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)x, CTRL, ROWS, 0xf, false);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)(x >> 32), CTRL, ROWS, 0xf, false);
    return x + ((u64)hi << 32 | lo);
}
__device__ __forceinline__ u64 wave_running(u64 x) {
    x = dpp_plus<0x111, 0xf>(x);   // from 1, 2, 4 and 8 lanes below within a row of 16
    x = dpp_plus<0x112, 0xf>(x);
    x = dpp_plus<0x114, 0xf>(x);
    x = dpp_plus<0x118, 0xf>(x);
    x = dpp_plus<0x142, 0xa>(x);   // a row's last lane to the next row
    return dpp_plus<0x143, 0xc>(x);   // lane 31 to the upper half
}
__device__ __forceinline__ u64 of_lane(u64 x, int lane) {
    return (u64)(uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(x >> 32), lane) << 32 | (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)x, lane);
}
__device__ __forceinline__ u64 wave_sum(u64 x) { return of_lane(wave_running(x), 63); }

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

struct Part { float top; int at, bin, count; u64 mass; };   // count and mass of all its bins
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

// kCopies histograms side by side, a lane's by its number, keep lanes that meet in
// a bin apart (256 rows of 65,536: 22 us, with one 43).
constexpr int kCopies = 4;
template <typename T> __global__ __launch_bounds__(kPartThreads) void parts_kernel(const SampleArgs a, const Work w, int bits) {
    __shared__ uint32_t count[kBins * kCopies];
    __shared__ u64 mass[kBins * kCopies];
    __shared__ double root[64];
    __shared__ float tops[kPartThreads / 64];
    __shared__ int ats[kPartThreads / 64];
    static_assert(kPartThreads == kBins, "a bin a thread");
    const int tid = threadIdx.x, lo = (blockIdx.x % w.parts) * w.length, hi = min(lo + w.length, a.vocab);
    const long n = blockIdx.x / w.parts;
    const T *x = static_cast<const T *>(a.logits) + n * a.stride;
    const Limits lim = limits_of(a, n);
#pragma unroll
    for (int i = 0; i < kCopies; ++i) {
        count[tid + i * kBins] = 0;
        mass[tid + i * kBins] = 0;
    }
    fill_roots(root, bits);
    float top = -__builtin_inff();
    int at = INT32_MAX;
    each_of<kPartThreads, 4>(x, lo, hi, [&](float y, int i) {
        if (y > top || (y == top && i < at)) {
            top = y;
            at = i;
        }
    });
    block_top(top, at, tops, ats);
    if (!(top > -__builtin_inff()) || !(lim.temperature > 0.f)) {
        if (tid == 0) w.part[blockIdx.x] = Part{top, at, 0, 0, 0};
        return;
    }
    const Row row = row_at(top, lim.temperature, bits, root);
    const int first = row.bin(top), copy = tid & (kCopies - 1);
    const auto count_all = [&](auto counts, auto weighs) {
        each_of<kPartThreads, 2>(x, lo, hi, [&](float y, int) {
            if (!counted(y)) return;
            const int b = (int)min((uint32_t)(first - row.bin(y)), (uint32_t)kBins - 1) * kCopies + copy;
            if constexpr (decltype(counts)::value) atomicAdd(&count[b], 1u);
            if constexpr (decltype(weighs)::value) atomicAdd(&mass[b], row.weight(y));
        });
    };
    if (lim.counts) count_all(std::true_type{}, std::false_type{});
    else if (lim.by_k) count_all(std::true_type{}, std::true_type{});
    else count_all(std::false_type{}, std::true_type{});
    __syncthreads();
    u64 c = 0, m = 0;
#pragma unroll
    for (int i = 0; i < kCopies; ++i) {
        c += count[tid * kCopies + i];
        m += mass[tid * kCopies + i];
    }
    if (lim.by_k) w.count[(long)blockIdx.x * kBins + tid] = (uint32_t)c;
    if (!lim.counts) w.mass[(long)blockIdx.x * kBins + tid] = m;
    __syncthreads();
    c = wave_sum(c);
    m = wave_sum(m);
    if ((tid & 63) == 0) {
        count[tid >> 6] = (uint32_t)c;
        mass[tid >> 6] = m;
    }
    __syncthreads();
    if (tid == 0) w.part[blockIdx.x] = Part{top, at, first, (int)(count[0] + count[1] + count[2] + count[3]), mass[0] + mass[1] + mass[2] + mass[3]};
}

// ---- second launch: the cut and the token --------------------------------------

struct Shared {
    uint32_t count[kFine];
    u64 mass[kFine];
    u64 list[kList], list_mass[kList];
    u64 few[kFew], few_mass[kFew], sorted[kFew], sorted_mass[kFew];
    uint32_t rank[kFew];
    double root[64];
    uint32_t digit[256];
    u64 digit_mass[256];
    u64 sums[kWaves], part_mass[kMostParts];
    double factor[kMostParts];
    int shift[kMostParts];
    u64 out[4];
    int listed, found;
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
            before = of_lane(incl - own, k);
            return i + k;
        }
        sum = of_lane(incl, 63);
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

// The least weights' sum that keeps top_p of all.
__device__ __forceinline__ u64 share_of(float top_p, u64 all) {
    return max(min((u64)__builtin_ceil((double)__builtin_fmaxf(top_p, 0.f) * (double)all), all), (u64)1);
}

// n <= kFew places with their weights put in order, into sh.sorted: each
// against the others, a quarter of them a thread.  BY_INDEX: in the order of
// indices.
template <bool BY_INDEX> __device__ __forceinline__ void sort_few(Shared &sh, const u64 *from, const u64 *weights, int n) {
    const int tid = threadIdx.x, mine = tid & (kFew - 1), lo = tid / kFew * (kFew / 4), hi = min(lo + kFew / 4, n);
    const auto order = [](u64 p) { return BY_INDEX ? (uint32_t)p : p; };
    if (tid < kFew) sh.rank[tid] = 0;
    __syncthreads();
    if (mine < n) {
        const u64 p = order(from[mine]);
        uint32_t r = 0;
#pragma unroll 8
        for (int i = lo; i < hi; ++i) r += order(from[i]) < p;
        if (r) atomicAdd(&sh.rank[mine], r);
    }
    __syncthreads();
    if (tid < n) {
        sh.sorted[sh.rank[tid]] = from[tid];
        sh.sorted_mass[sh.rank[tid]] = weights[tid];
    }
    __syncthreads();
}

// How many of sh.sorted's first n stand before the running count (or sum of
// weights, BY_MASS) is at least `want`, and the one with which it is; `upto`: the
// sum of their weights.  By one wave, four a lane.
template <bool BY_MASS> __device__ __forceinline__ int few_reaching(const Shared &sh, int n, u64 want, u64 &upto) {
    const int lane = threadIdx.x & 63;
    u64 y[4], s = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        y[i] = 4 * lane + i < n ? sh.sorted_mass[4 * lane + i] : 0;
        s += y[i];
    }
    u64 run = wave_running(s) - s;
    int mine = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int k = 4 * lane + i;
        mine += k < n && (BY_MASS ? run < want : (u64)k < want);
        run += y[i];
    }
    const int all = (int)wave_sum((u64)mine);
    u64 kept = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (4 * lane + i < all) kept += y[i];
    upto = wave_sum(kept);
    return all;
}

// Among the places each() goes over, with keys in [lo, hi], the first at which the
// running count (or sum of weights, BY_MASS) is at least `want`; `upto`: the sum of
// weights up to it and its own.  A histogram of 256 equal pieces of the keys says in
// which piece it lies, and so on until few are left, which are put in order; equal
// keys are told apart by index.  BY_INDEX: the index is the key.  each(f) calls
// f(place, a function that gives its weight).  ~0 where there is no place.
template <typename T, bool BY_MASS, bool BY_INDEX, typename Each>
__device__ u64 nth(Shared &sh, const Each &each, uint32_t lo, uint32_t hi, int V, u64 want, u64 &upto) {
    const int tid = threadIdx.x;
    bool tie = BY_INDEX;             // the index is looked at
    uint32_t equal = 0;              // the key of those that are
    u64 less = 0;                    // weights of what lies before [lo, hi]
    for (;;) {
        const uint32_t width = hi - lo;
        const int s = max(0, 24 - __builtin_clz(width | 1));
        const auto piece = [&](u64 p) -> int {     // of the range, or -1
            if (!BY_INDEX && tie && place_key<T>(p) != equal) return -1;
            const uint32_t k = (tie ? (uint32_t)p : place_key<T>(p)) - lo;
            return k <= width ? (int)(k >> s) : -1;
        };
        if (tid < 256) {
            sh.digit[tid] = 0;
            sh.digit_mass[tid] = 0;
        }
        if (tid == 0) sh.found = 0;
        __syncthreads();
        each([&](u64 p, auto weight) {
            const int d = piece(p);
            if (d >= 0) {
                atomicAdd(&sh.digit[d], 1u);
                atomicAdd(&sh.digit_mass[d], weight());
            }
        });
        __syncthreads();
        if (tid < 64) {
            u64 before, sum = 0;
            int d;
            if constexpr (BY_MASS) d = first_reaching(sh.digit_mass, 256, want, before);
            else d = first_reaching(sh.digit, 256, want, before);
            if (d == 256) {          // sums that differ in the last place: the last piece that has some
                for (int i = 192; i >= 0 && d == 256; i -= 64) {
                    const u64 some = __ballot(sh.digit[i + tid] > 0);
                    if (some) d = i + 63 - __builtin_clzll(some);
                }
                d = d == 256 ? 0 : d;
                before = BY_MASS ? before - sh.digit_mass[d] : before - sh.digit[d];
            }
            for (int i = tid; i < d; i += 64) sum += sh.digit_mass[i];
            sum = wave_sum(sum);
            if (tid == 0) {
                sh.out[0] = d;
                sh.out[1] = want - min(before, want);
                sh.out[2] = sum;
            }
        }
        __syncthreads();
        const int d = (int)sh.out[0], some = (int)sh.digit[d];
        want = sh.out[1];
        less += sh.out[2];
        if (some == 0) {
            upto = less;
            return ~0ull;
        }
        if (some <= kFew) {
            each([&](u64 p, auto weight) {
                if (piece(p) == d) {
                    const int at = atomicAdd(&sh.found, 1);
                    sh.few[at] = p;
                    sh.few_mass[at] = weight();
                }
            });
            __syncthreads();
            sort_few<BY_INDEX>(sh, sh.few, sh.few_mass, some);
            if (tid < 64) {
                u64 sum;
                const int k = few_reaching<BY_MASS>(sh, some, want, sum);
                if (tid == 0) {
                    sh.out[0] = sh.sorted[max(k, 1) - 1];
                    sh.out[1] = sum;
                }
            }
            __syncthreads();
            const u64 p = sh.out[0];
            upto = less + sh.out[1];
            __syncthreads();
            return p;
        }
        __syncthreads();
        lo += (uint32_t)d << s;
        hi = lo + min(hi - lo, (1u << s) - 1);   // the piece's end itself may lie past 2^32
        if (s == 0) {                // one key, and more than a few that have it
            equal = lo;
            tie = true;
            lo = 0;
            hi = (uint32_t)V - 1;
        }
    }
}

// The last key of [lo, hi) for which holds() is true; it is true at lo and, once
// false, stays false.  By one wave.
template <typename Holds> __device__ __forceinline__ uint32_t last_key(uint32_t lo, uint32_t hi, const Holds &holds) {
    const int lane = threadIdx.x & 63;
    while (hi - lo > 1) {
        const uint32_t step = (hi - lo + 63) / 64;
        const u64 k = (u64)lo + (u64)step * lane;
        const int last = 63 - __builtin_clzll(__ballot(k < hi && (lane == 0 || holds((uint32_t)k))));
        hi = (uint32_t)min((u64)lo + (u64)step * (last + 1), (u64)hi);
        lo += step * last;
    }
    return lo;
}
constexpr uint32_t kLowest = 0xff7fffffu;   // the key of the lowest finite number: the last that counts

// The row's logits in [from, to] into sh.list, with their weights; as many as the
// caller has counted.
template <typename T> __device__ __forceinline__ void gather(Shared &sh, const Row &row, const T *x, int V, float from, float to) {
    constexpr int N = 16 / (int)sizeof(T), AHEAD = 4;
    const int tid = threadIdx.x, head = min(V, (int)((0 - reinterpret_cast<uintptr_t>(x)) % 16 / sizeof(T))), wide = (V - head) / N;
    const auto take = [&](int i) {
        const float y = value(x, i);
        if (y >= from && y <= to) {
            const int at = atomicAdd(&sh.listed, 1);
            if (at < kList) sh.list[at] = place_of<T>(y, i);
        }
    };
    if (tid == 0) sh.listed = 0;
    __syncthreads();
    if (tid < head) take(tid);
    for (int v = tid; v < wide; v += AHEAD * kThreads) {
        u32x4 w[AHEAD];
#pragma unroll
        for (int k = 0; k < AHEAD; ++k) w[k] = *reinterpret_cast<const u32x4 *>(x + head + (long)min(v + k * kThreads, wide - 1) * N);
        uint32_t in = 0;             // few are taken: one look at 32 of them
#pragma unroll
        for (int k = 0; k < AHEAD; ++k)
#pragma unroll
            for (int e = 0; e < N; ++e) {
                float y;
                if constexpr (N == 4) y = __uint_as_float(w[k][e]);
                else y = __uint_as_float(e & 1 ? w[k][e / 2] & 0xffff0000u : w[k][e / 2] << 16);
                in |= (uint32_t)(y >= from && y <= to) << (k * N + e);
            }
        while (in) {
            const int e = __builtin_ctz(in);
            in &= in - 1;
            if (v + e / N * kThreads < wide) take(head + (v + e / N * kThreads) * N + e % N);
        }
    }
    const int tail = head + wide * N;
    if (tail + tid < V) take(tail + tid);
    __syncthreads();
    for (int i = tid; i < min(sh.listed, kList); i += kThreads) sh.list_mass[i] = row.weight(place_value<T>(sh.list[i]));
    __syncthreads();
}

// The cut of a row whatever its logits, from passes over all of it: for rows
// with more logits in the cut's bin than the list holds (thousands of equal
// ones, weights so flat that a cut lies far down).  One workgroup's latency: a row of
// 131,072 normal logits at temperature 5 with top_p 0.9 takes 262 us, 256 such rows
// 449; equal logits, which meet in one bin's atomics, 1.5 ms.
template <typename T> __device__ u64 cut_of_whole_row(Shared &sh, const Row &row, const Limits &lim, const T *x, int V) {
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
        if (!counted(y)) continue;
        const int b = bin(y);
        atomicAdd(&sh.count[b], 1u);
        atomicAdd(&sh.mass[b], row.weight(y));
    }
    __syncthreads();
    const auto cut_in = [&](int b, auto by_mass, u64 want, u64 &upto) {
        const auto each = [&](auto f) {
            for (int i = tid; i < V; i += kThreads) {
                const float y = value(x, i);
                if (counted(y) && bin(y) == b) f(place_of<T>(y, i), [&] { return row.weight(y); });
            }
        };
        return nth<T, decltype(by_mass)::value, false>(sh, each, cut_key<T>(key_of(row.top)), cut_key<T>(kLowest), V, want, upto);
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
        const u64 want = share_of(lim.top_p, block_sum(sh, s) + upto);
        const int b = block_reaching(sh, sh.mass, kFine, want, before);
        cut = min(cut, cut_in(min(b, kFine - 1), std::true_type{}, want - min(before, want), upto));
    }
    return cut;
}

template <typename T> __global__ __launch_bounds__(kThreads) void choose_kernel(const SampleArgs a, const Work w, int bits) {
    __shared__ Shared sh;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, V = a.vocab;
    const long n = blockIdx.x;
    const T *x = static_cast<const T *>(a.logits) + n * a.stride;
    const Limits lim = limits_of(a, n);
    // the parts' bins, one a thread of a quarter of the parts each: asked for before
    // anything else, as they come from far
    constexpr int QUARTER = kThreads / kBins, EACH = kMostParts / QUARTER;
    const int own_bin = tid & (kBins - 1), own_part = tid / kBins;
    uint32_t part_count[EACH];
    u64 part_mass[EACH];
#pragma unroll
    for (int k = 0; k < EACH; ++k) {
        const long from = (n * w.parts + min(own_part + k * QUARTER, w.parts - 1)) * kBins + own_bin;
        part_count[k] = lim.by_k ? w.count[from] : 0;
        part_mass[k] = lim.counts ? 0 : w.mass[from];
    }
    // a part a lane
    const Part mine = lane < w.parts ? w.part[n * w.parts + lane] : Part{-__builtin_inff(), INT32_MAX, 0, 0, 0};
    float top = mine.top;
    int at = mine.at;
#pragma unroll
    for (int m = 32; m >= 1; m >>= 1) {
        const float y = __shfl_xor(top, m, 64);
        const int j = __shfl_xor(at, m, 64);
        if (y > top || (y == top && j < at)) {
            top = y;
            at = j;
        }
    }
    if (!(top > -__builtin_inff()) || !(lim.temperature > 0.f)) {   // no logit at all, or the largest
        if (tid == 0) {
            const bool none = !(top > -__builtin_inff());
            if (a.tokens) a.tokens[n] = none ? -1 : at;
            w.row[n] = Chosen{0, 0, top, at, none ? kNothing : kLargest, 0};
        }
        return;
    }
    fill_roots(sh.root, bits);
    const Row row = row_at(top, lim.temperature, bits, sh.root);
    const int first = row.bin(top);
    const auto bin = [&](float y) { return (int)min((uint32_t)(first - row.bin(y)), (uint32_t)kBins - 1); };
    if (tid < kBins) {
        sh.count[tid] = 0;
        sh.mass[tid] = 0;
    }
    __syncthreads();
    // the parts' bins and weights against the row's largest
    if (tid < kMostParts) {
        sh.shift[tid] = min(first - mine.bin, kBins - 1);
        sh.factor[tid] = mine.top > -__builtin_inff() ? row.real(mine.top) / row.one : -1.0;   // -1: nothing there
    }
    __syncthreads();
    if (lim.by_k || lim.by_p) {
        // the last bin has what is left of the sums
#pragma unroll
        for (int k = 0; k < EACH; ++k) {
            const int p = own_part + k * QUARTER;
            if (p >= w.parts || sh.factor[p] < 0.0) continue;
            const int to = own_bin + sh.shift[p];
            if (to >= kBins - 1) continue;
            if (part_count[k]) atomicAdd(&sh.count[to], part_count[k]);
            if (part_mass[k]) atomicAdd(&sh.mass[to], (u64)__builtin_rint((double)part_mass[k] * sh.factor[p]));
        }
        __syncthreads();
        if (wave == 0) {
            u64 cs = 0, ms = 0;
            for (int i = lane; i < kBins - 1; i += 64) {
                cs += sh.count[i];
                ms += sh.mass[i];
            }
            cs = wave_sum(cs);
            ms = wave_sum(ms);
            const u64 call = wave_sum(sh.factor[lane] < 0.0 ? 0 : (u64)mine.count);
            const u64 mall = wave_sum(lim.counts || sh.factor[lane] < 0.0 ? 0 : (u64)__builtin_rint((double)mine.mass * sh.factor[lane]));
            if (lane == 0) {
                sh.count[kBins - 1] = (uint32_t)(call - cs);
                sh.mass[kBins - 1] = mall > ms ? mall - ms : 0;
            }
        }
        __syncthreads();
    }

    u64 cut = ~0ull;                 // the last place that is kept
    if (lim.by_m) {                  // the smallest number whose weight is not below the limit
        if (wave == 0) {
            const double least = (double)lim.min_p * row.one;
            const uint32_t k = last_key(key_of(top), kLowest + 1, [&](uint32_t k) { return row.real(of_key(k)) >= least; });
            if (lane == 0) sh.out[0] = last_of_key<T>(k);
        }
        __syncthreads();
        cut = sh.out[0];
        __syncthreads();
    }
    // the smallest logit of bins up to b (b >= 0)
    const auto end_of = [&](int b) {
        if (b >= kBins - 1) return kLowest;
        return last_key(key_of(top), kLowest + 1, [&](uint32_t k) { return bin(of_key(k)) <= b; });
    };
    const auto listed_each = [&](auto f) {
        const int some = sh.listed;
        for (int i = tid; i < some; i += kThreads) f(sh.list[i], [&] { return sh.list_mass[i]; });
    };
    const uint32_t key_lo = cut_key<T>(key_of(top));

    bool whole = false;              // the list cannot hold a cut's bin
    u64 total = 0;                   // of the weights kept
    if (lim.counts) {
        // few are kept: all logits up to the bin of the k-th
        u64 before;
        const int b = min(block_reaching(sh, sh.count, kBins, (u64)lim.top_k, before), kBins - 1);
        whole = block_sum(sh, tid <= b ? sh.count[tid] : 0) > (u64)kList;
        if (!whole) {
            const uint32_t end = end_of(b);
            gather(sh, row, x, V, of_key(end), top);
            const int some = sh.listed;
            if (some <= kFew) {
                sort_few<false>(sh, sh.list, sh.list_mass, some);
                if (wave == 0) {
                    u64 all, upto;
                    int keep = few_reaching<false>(sh, some, (u64)lim.top_k, all);
                    if (lim.by_p) keep = few_reaching<true>(sh, keep, share_of(lim.top_p, all), upto);
                    if (lim.by_m)
                        while (sh.sorted[keep - 1] > cut) --keep;
                    few_reaching<false>(sh, keep, (u64)keep, upto);
                    if (lane == 0) {
                        sh.out[0] = keep;
                        sh.out[1] = upto;
                    }
                }
                __syncthreads();
                const int keep = (int)sh.out[0];
                total = sh.out[1];
                cut = sh.sorted[keep - 1];
                if (a.tokens && tid < keep) {
                    // the running sum by index of every logit kept
                    const u64 want = min((u64)((double)a.uniform[n] * (double)total), total - 1);
                    const uint32_t i = (uint32_t)sh.sorted[tid];
                    const u64 own = sh.sorted_mass[tid];
                    u64 below = 0;
#pragma unroll 4
                    for (int j = 0; j < keep; ++j)
                        if ((uint32_t)sh.sorted[j] < i) below += sh.sorted_mass[j];
                    if (below <= want && below + own > want) a.tokens[n] = (int)i;
                }
            } else {
                u64 all, upto;
                if (some > lim.top_k) {
                    cut = min(cut, nth<T, false, false>(sh, listed_each, key_lo, cut_key<T>(end), V, (u64)lim.top_k, all));
                } else {   // all that are listed; others may follow
                    cut = min(cut, last_of_key<T>(end));
                    u64 s = 0;
                    listed_each([&](u64, auto weight) { s += weight(); });
                    all = block_sum(sh, s);
                }
                if (lim.by_p) cut = min(cut, nth<T, true, false>(sh, listed_each, key_lo, cut_key<T>(end), V, share_of(lim.top_p, all), upto));
                u64 s = 0;
                listed_each([&](u64 p, auto weight) { s += p <= cut ? weight() : 0; });
                total = block_sum(sh, s);
                if (a.tokens) {
                    const auto kept_each = [&](auto f) {
                        listed_each([&](u64 p, auto weight) {
                            if (p <= cut) f(p, weight);
                        });
                    };
                    const u64 want = min((u64)((double)a.uniform[n] * (double)total), total - 1) + 1;
                    const u64 p = nth<T, true, true>(sh, kept_each, 0, (uint32_t)V - 1, V, want, upto);
                    if (tid == 0) a.tokens[n] = (int)(uint32_t)p;
                }
            }
            if (tid == 0) w.row[n] = Chosen{cut, total, top, at, kDrawn, 0};
            return;
        }
    }
    int edge = kBins;                // the bin that the cut goes through: those before it are kept whole
    int listed = -1;                 // the bin whose logits the list holds
    uint32_t list_lo = 0, list_hi = 0;   // and their keys
    if (!lim.counts) {
        const auto list = [&](int b) {   // true where it holds them all
            if (listed == b) return true;
            if (wave < 2) {
                const uint32_t k = wave == 0 ? end_of(b) : b > 0 ? end_of(b - 1) + 1 : key_of(top);
                if (lane == 0) sh.out[wave] = k;
            }
            __syncthreads();
            list_hi = (uint32_t)sh.out[0];
            list_lo = (uint32_t)sh.out[1];
            __syncthreads();
            gather(sh, row, x, V, of_key(list_hi), of_key(list_lo));
            listed = b;
            return sh.listed <= kList;
        };
        const auto cut_in = [&](auto by_mass, u64 want, u64 &upto) {
            return nth<T, decltype(by_mass)::value, false>(sh, listed_each, cut_key<T>(list_lo), cut_key<T>(list_hi), V, want, upto);
        };
        u64 before, upto = 0;
        int last = kBins;
        if (lim.by_k) {
            last = block_reaching(sh, sh.count, kBins, (u64)lim.top_k, before);
            if (last < kBins) {
                whole = !list(last);
                if (!whole) {
                    cut = min(cut, cut_in(std::false_type{}, (u64)lim.top_k - before, upto));
                    edge = last;
                }
            }
        }
        const int limit = lim.by_m ? bin(place_value<T>(cut)) : kBins;   // the bin of min_p's own number
        if (lim.by_p && !whole) {
            const u64 want = share_of(lim.top_p, block_sum(sh, tid < last && tid < kBins ? sh.mass[tid] : 0) + upto);
            const int b = min(block_reaching(sh, sh.mass, kBins, want, before), kBins - 1);
            if (b <= limit) whole = !list(b);
            if (b <= limit && !whole) {
                cut = min(cut, cut_in(std::true_type{}, want - min(before, want), upto));
                edge = min(edge, b);
            }
        }
        edge = min(edge, limit);
        if (!whole && edge < kBins) whole = !list(edge);
    }
    if (whole) {
        __syncthreads();
        const u64 least = cut;
        cut = min(lim.by_m ? least : ~0ull, cut_of_whole_row(sh, row, lim, x, V));
    }

    const auto kept = [&](float y, int i) -> u64 { return y == y && place_of<T>(y, i) <= cut ? row.weight(y) : 0; };
    int lo = 0, hi = V;
    u64 want = 0;
    if (!whole) {
        // what every part keeps: its bins before the cut's, and its share of the list
        if (tid < kMostParts) sh.part_mass[tid] = 0;
        __syncthreads();
        if (listed >= 0)
            listed_each([&](u64 p, auto weight) {
                if (p <= cut) atomicAdd(&sh.part_mass[(uint32_t)p / (uint32_t)w.length], weight());
            });
#pragma unroll
        for (int k = 0; k < EACH; ++k) {
            const int p = own_part + k * QUARTER;
            // A part whose largest logit is below half a unit of the row (or has none) holds
            // nothing that could be drawn, though its own sum, in finer units, may round to
            // one and more.  In any other part that has logits before the cut's bin its
            // largest is one of them, so a part with a sum has a logit that weighs.
            if (p >= w.parts || !(sh.factor[p] * row.one > 0.5)) continue;
            const u64 s = wave_sum(edge == kBins || min(own_bin + sh.shift[p], kBins - 1) < edge ? part_mass[k] : 0);
            if (lane == 0 && s) atomicAdd(&sh.part_mass[p], (u64)__builtin_rint((double)s * sh.factor[p]));
        }
        __syncthreads();
        if (wave == 0) {
            const u64 own = sh.part_mass[lane], incl = wave_running(own), all = of_lane(incl, 63);
            u64 to = 0;
            if (a.tokens) to = min((u64)((double)a.uniform[n] * (double)all), all - 1);
            const u64 past = __ballot(incl > to);
            const int p = past ? __builtin_ctzll(past) : 0;
            const u64 rest = to - of_lane(incl - own, p);
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
        if (tid == 0) w.row[n] = Chosen{cut, total, top, at, kDrawn, 0};
        if (!a.tokens) return;
    }
    // by sixteenths of what is left of the row
    for (bool firstly = whole; firstly || hi - lo > 64; firstly = false) {
        const int each = (hi - lo + kWaves - 1) / kWaves, from = min(lo + wave * each, hi), to = min(from + each, hi);
        u64 s = 0;
        constexpr int AHEAD = 8;
        for (int i = from + lane; i < to; i += 64 * AHEAD) {
            float y[AHEAD];
#pragma unroll
            for (int k = 0; k < AHEAD; ++k) y[k] = value(x, min(i + 64 * k, to - 1));
#pragma unroll
            for (int k = 0; k < AHEAD; ++k)
                if (i + 64 * k < to) s += kept(y[k], i + 64 * k);
        }
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
        if (sh.sums[part] <= want) {   // sums of parts and of their logits may differ in the last place: the last one that weighs
            while (part > 0 && sh.sums[part] == 0) --part;
            want = max(sh.sums[part], (u64)1) - 1;
        }
        lo = min(lo + part * each, hi);
        hi = min(lo + each, hi);
        __syncthreads();
    }
    if (wave == 0) {
        const u64 own = lo + lane < hi ? kept(value(x, lo + lane), lo + lane) : 0, incl = wave_running(own);
        const u64 past = __ballot(incl > want), some = __ballot(own > 0);   // some: never none
        if (lane == 0) a.tokens[n] = lo + (past ? __builtin_ctzll(past) : 63 - __builtin_clzll(some | 1));
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
    fill_roots(root, bits);
    __syncthreads();
    const Row row = row_at(c.top, a.temperature ? a.temperature[n] : 1.f, bits, root);
    const double f = 1.0 / (double)c.total;
    for (int i = lo + threadIdx.x; i < hi; i += kPartThreads) {
        const float y = value(x, i);
        probs[i] = y == y && place_of<T>(y, i) <= c.cut ? (float)(row.real(y) * f) : 0.f;
    }
}

size_t round_up(size_t n) { return (n + 255) / 256 * 256; }

// Parts of a row: enough workgroups for the chip, of 4096 logits or more; of
// 8192 at most, as the token's part is gone through again by one workgroup.
void lay_out(Work &w, int rows, int vocab, void *workspace, size_t &bytes) {
    const long most = std::min<long>(kMostParts, (vocab + 4095) / 4096);
    w.parts = (int)std::max<long>(1, std::min<long>(most, std::max<long>((1024 + rows - 1) / rows, vocab / 8192)));
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

bool sample_fits(int rows, int vocab) {
    Work w{};
    size_t bytes = 0;
    lay_out(w, rows, vocab, nullptr, bytes);
    return (size_t)rows <= UINT32_MAX / kThreads && (size_t)rows * w.parts <= UINT32_MAX / kPartThreads;
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
