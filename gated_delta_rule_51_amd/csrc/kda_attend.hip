// Causal attention over a paged cache of 8-bit keys and values.
//
//   o_j = sum_i p_ij v_i / sum_i p_ij,  p_ij = exp(scale q_j . k_i - m_j),  i <= last_j
//
// with a running reference m (softmax's value does not depend on it).  A query
// is a column: the g query heads that share a key head, times the tokens, are
// the columns of S^T = K Q^T and O^T = V^T P^T, so keys and values are read
// once for all of them and both are the matrix cores' A operand.
//
// Fragments come straight from memory, 16 bytes a lane, without LDS: the rows
// of a 64-key tile are numbered so that the four S^T tiles leave lane group
// l / 16 with the scores of its keys 16 (l / 16) .. + 15, which is what the B
// operand of the second product wants from it, and so that its share of V^T is
// 16 consecutive tokens of one channel (values are stored with tokens side by
// side).  Head channels are taken in the order 64 j + 16 (l / 16) + e for the
// same reason.  e4m3 widens to bf16 exactly, and the block's power-of-two scale
// goes in with it.
//
// Arithmetic: bf16 queries are operands as they are.  p goes in as the sum of two
// bf16 terms (16 bits) for single tokens and drafts, where memory leaves time for
// it (64 tokens 112.2 us with one term and 112.5 with two, drafts 106 and 108, in two
// column tiles 93 and 96; the error falls from 2.1e-3 to 1.66e-3, of which the
// output's own rounding is 1.65e-3), and rounded to bf16, for its sum too, in the
// kernel for prompts, whose registers a second term overflows (638 us with one,
// 1241 with two).  fp32 queries and their p go in as the sum of three bf16 terms.
// Scores, sums and outputs accumulate in fp32.
//
// Work is cut into (request, columns, chunk of keys) units over a fixed number
// of places: the chunk length follows from the lengths on the device, such that
// the places always suffice and hold about equal work.  Chunks of one column
// are joined by a second launch.
//
// Bound by HBM for single tokens and drafts (one token of 64 requests of 100 to
// 16,000 tokens, 4 heads x 128: 547 MB in 112.5 us; four drafts of 128 requests, 16
// heads x 64: 108 us, 5.1 TB/s), by vector instructions, nearly five beside each
// matrix one, for prompts (4 of 2000 to 4096 tokens, 32 over 8 heads x 128: 624 to 638
// us, 896 TFLOP/s, 73% of what a large bf16 product reaches).
#include <algorithm>

#include "kda_device.h"
#include "kda_internal.h"

namespace kda {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

constexpr int kWaves = 4, kThreads = 64 * kWaves;
constexpr float kNone = -1e30f;   // a reference below every score

// How a call is laid out over the chip.  Columns of a workgroup: SPLIT kernels
// give their four waves the same 16 NT columns and every fourth key tile,
// the others each wave 16 NT of its own.
struct Layout {
    int nt;
    int keys;        // of a tile
    bool split;
    int cols;        // of a workgroup
    long units;      // (request, columns) pairs, at most
    long places;     // units and room for chunks
};

Layout layout_of(int num_seqs, int total_tokens, int q_heads, int heads, bool io_bf16) {
    Layout y{};
    const long g = q_heads / heads, columns = (long)total_tokens * g, each = num_seqs ? (columns + num_seqs - 1) / num_seqs : 0;
    y.nt = each <= 16 ? 1 : each <= 32 || !io_bf16 ? 2 : 4;
    y.split = each <= 32;
    y.keys = y.split ? 64 : 32;
    y.cols = 16 * y.nt * (y.split ? 1 : kWaves);
    y.units = columns / y.cols + num_seqs;
    // Prompts are cut where their undivided units are fewer than two workgroups a CU.
    // Cutting lets uneven contexts end together (6 prompts of 200 to 700 tokens behind up
    // to 16,000, 328 workgroups: 410 us cut, 649 whole) and costs even ones the join (2 of
    // 1000 to 1600, 376 workgroups: 156 and 114; 8 of up to 700, 464: 153 and 93); from 512 on whole was faster throughout
    // (16 of 50 to 500 behind up to 2000, 656: 234 and 145; 3 of 500 to 2000 behind up to
    // 8000, 552: 441 and 415).  Room for chunks: with half of 1024 the six prompts take
    // 495 us, with twice that 454.
    long more = 0;
    if (y.split) more = std::max<long>((768 + heads - 1) / heads, y.units / 4);
    else if (y.units * heads < 512) more = (1024 + heads - 1) / heads;
    y.places = y.units + more;
    static_assert(16 * 4 * kWaves <= 256, "a column's number has 8 bits");
    return y;
}

struct Plan {
    int units, places, least;   // least: tiles of a chunk
    int *info;                  // [tokens, query heads, 2]: place of a column's first chunk; how many it has, and the
                                // column's number there in the low 8 bits
    uint32_t *starts;           // [0]: chunk length; [1 + n]: first place of request n, the last: all places; or NULL
    float *sums;                // [places, heads, cols, 2]: m, l
    float *parts;               // [places, heads, cols, d]
};

// Up to this many requests every workgroup finds its place from the lengths by
// itself, a request a thread, which takes about a microsecond; for more a launch
// of one workgroup before them writes down where each request's places begin (1024
// requests of 50 to 600 tokens over 8 heads 204 us, with every workgroup by itself
// 281; 64 requests 115 with it, 112 without).
constexpr int kFindOwn = kThreads;
size_t starts_bytes(int num_seqs) { return num_seqs <= kFindOwn ? 0 : ((size_t)num_seqs * 4 + 8 + 255) / 256 * 256; }
size_t info_bytes(long columns) { return ((size_t)columns * 8 + 255) / 256 * 256; }

__device__ __forceinline__ uint32_t wave_sum(uint32_t x) {
#pragma unroll
    for (int m = 32; m >= 1; m >>= 1) x += __shfl_xor(x, m, 64);
    return x;
}
__device__ __forceinline__ unsigned long long wave_sum(unsigned long long x) {
#pragma unroll
    for (int m = 32; m >= 1; m >>= 1) x += __shfl_xor(x, m, 64);
    return x;
}

struct Request { int begin, length, total, units, tiles; };

__device__ __forceinline__ Request request_of(const AttendArgs &a, int n, int g, int cols, int keys) {
    Request r;
    r.begin = max(a.cu_seqlens[n], 0);
    r.length = max(min(a.cu_seqlens[n + 1], a.total_tokens) - r.begin, 0);
    const int row = a.indices[n];
    const long most = (long)a.max_blocks << a.block_shift;
    r.total = (unsigned)row < (unsigned)a.rows ? (int)min((long)max(a.kv_totals[n], 0), most) : 0;
    r.units = (int)(((long)r.length * g + cols - 1) / cols);
    r.tiles = (int)(((long)r.total + keys - 1) / keys);
    return r;
}

struct Unit { int n, column, chunk, chunks, length; };   // column: index of the unit's columns; length: tiles of a chunk

// Places of request r, and its chunks.
__device__ __forceinline__ uint32_t places_of(const Request &r, int length, int &chunks) {
    chunks = max(1, (r.tiles + length - 1) / length);
    return (uint32_t)r.units * chunks;
}

constexpr int kPlanThreads = 1024, kPlanWaves = kPlanThreads / 64;
__global__ __launch_bounds__(kPlanThreads) void plan_kernel(const AttendArgs a, const Plan plan, int cols, int keys) {
    __shared__ unsigned long long work[kPlanWaves];
    __shared__ uint32_t part[kPlanWaves];
    const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63, g = a.q_heads / a.heads;
    int length = INT32_MAX / 2;
    if (plan.places > plan.units) {
        unsigned long long w = 0;
        for (int n = tid; n < a.num_seqs; n += kPlanThreads) {
            const Request r = request_of(a, n, g, cols, keys);
            w += (unsigned long long)r.units * r.tiles;
        }
        w = wave_sum(w);
        if (lane == 0) work[wave] = w;
        __syncthreads();
        w = 0;
#pragma unroll
        for (int i = 0; i < kPlanWaves; ++i) w += work[i];
        const unsigned long long room = plan.places - plan.units;
        length = (int)max((unsigned long long)plan.least, (w + room - 1) / room);
    }
    if (tid == 0) plan.starts[0] = (uint32_t)length;
    uint32_t before = 0;
    for (int n0 = 0; n0 < a.num_seqs; n0 += kPlanThreads) {
        const int n = n0 + tid;
        int chunks;
        uint32_t take = 0;
        if (n < a.num_seqs) take = places_of(request_of(a, n, g, cols, keys), length, chunks);
        uint32_t incl = take;
#pragma unroll
        for (int m = 1; m < 64; m <<= 1) {
            const uint32_t y = __shfl_up(incl, m, 64);
            if (lane >= m) incl += y;
        }
        if (lane == 63) part[wave] = incl;
        __syncthreads();
        incl += before;
#pragma unroll
        for (int w = 0; w < kPlanWaves; ++w) {
            if (w < wave) incl += part[w];
            before += part[w];
        }
        if (n < a.num_seqs) plan.starts[1 + n] = incl - take;
        __syncthreads();
    }
    if (tid == 0) plan.starts[1 + a.num_seqs] = before;
}

// What place p stands for, from the places' begins: a search 64 ways a step by
// each wave for itself.
__device__ Unit planned_unit_of(const AttendArgs &a, const Plan &plan, int p, int g, int cols, int keys) {
    const int lane = threadIdx.x & 63;
    const uint32_t *starts = plan.starts + 1;
    Unit u{-1, 0, 0, 1, (int)plan.starts[0]};
    if ((uint32_t)p >= starts[a.num_seqs]) return u;
    int lo = 0, num = a.num_seqs;
    while (num > 1) {
        const int step = (num + 63) / 64, i = lane * step;
        const unsigned long long m = __ballot(i < num && starts[lo + min(i, num - 1)] <= (uint32_t)p);
        const int k = (63 - __builtin_clzll(m | 1)) * step;
        lo += k;
        num = min(step, num - k);
    }
    places_of(request_of(a, lo, g, cols, keys), u.length, u.chunks);
    u.n = lo;
    u.column = (int)(p - starts[lo]) / u.chunks;
    u.chunk = (int)(p - starts[lo]) % u.chunks;
    return u;
}

// The same (n < 0: nothing) from the lengths.
__device__ Unit unit_of(const AttendArgs &a, const Plan &plan, int p, int g, int cols, int keys) {
    __shared__ unsigned long long work[kWaves];
    __shared__ uint32_t part[kWaves];
    __shared__ int found[4];
    const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
    Unit u{-1, 0, 0, 1, INT32_MAX / 2};
    if (plan.places > plan.units) {
        unsigned long long w = 0;
        for (int n = tid; n < a.num_seqs; n += kThreads) {
            const Request r = request_of(a, n, g, cols, keys);
            w += (unsigned long long)r.units * r.tiles;
        }
        w = wave_sum(w);
        if (lane == 0) work[wave] = w;
        __syncthreads();
        w = work[0] + work[1] + work[2] + work[3];
        const unsigned long long room = plan.places - plan.units;
        u.length = (int)max((unsigned long long)plan.least, (w + room - 1) / room);
    }
    if (tid == 0) found[0] = -1;
    __syncthreads();
    uint32_t before = 0;
    for (int n0 = 0; n0 < a.num_seqs; n0 += kThreads) {
        const int n = n0 + tid;
        uint32_t take = 0;
        int chunks = 1;
        if (n < a.num_seqs) {
            take = places_of(request_of(a, n, g, cols, keys), u.length, chunks);
        }
        uint32_t incl = take;
#pragma unroll
        for (int m = 1; m < 64; m <<= 1) {
            const uint32_t y = __shfl_up(incl, m, 64);
            if (lane >= m) incl += y;
        }
        if (lane == 63) part[wave] = incl;
        __syncthreads();
        uint32_t all = 0;
        incl += before;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) {
            if (w < wave) incl += part[w];
            all += part[w];
        }
        if ((uint32_t)p < incl && (uint32_t)p >= incl - take) {
            found[0] = n;
            found[1] = (int)(p - (incl - take)) / chunks;
            found[2] = (int)(p - (incl - take)) % chunks;
            found[3] = chunks;
        }
        before += all;
        __syncthreads();
        if (before > (uint32_t)p) break;
    }
    u.n = found[0];
    u.column = found[1];
    u.chunk = found[2];
    u.chunks = found[3];
    return u;
}

// The same for up to 64 requests and undivided keys, the units with the most keys
// first, so that the last workgroups to start are the shortest (four prompts of
// 2000 to 4096 tokens: 686 -> 669 us).  By each wave for itself, a request a
// lane: a search for the number of keys that just the units before p pass.
__device__ Unit longest_unit_of(const AttendArgs &a, int p, int g, int cols, int keys) {
    const int lane = threadIdx.x & 63;
    Request r{};
    if (lane < a.num_seqs) r = request_of(a, lane, g, cols, keys);
    const int before = r.total - r.length;
    // of the request's units, those that see more than x keys
    const auto past = [&](int x) {
        const long tokens = max((long)x - before, 0l);
        return r.units - (int)min((long)r.units, tokens * g / cols);
    };
    int hi = r.total + cols, lo = before;   // none see more; all do
#pragma unroll
    for (int m = 32; m >= 1; m >>= 1) {
        hi = max(hi, __shfl_xor(hi, m, 64));
        lo = min(lo, __shfl_xor(lo, m, 64));
    }
    Unit u{-1, 0, 0, 1, INT32_MAX / 2};
    if (p >= (int)wave_sum((uint32_t)r.units)) return u;
    while ((uint32_t)hi - (uint32_t)lo > 1) {   // the least x that at most p units pass; apart by up to 2^32
        const int x = lo + (int)(((uint32_t)hi - (uint32_t)lo) / 2);
        if ((int)wave_sum((uint32_t)past(x)) <= p) hi = x;
        else lo = x;
    }
    const int mine = past(hi), at = past(hi - 1) - mine;   // in front; at this number of keys
    uint32_t incl = at;
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) {
        const uint32_t y = __shfl_up(incl, m, 64);
        if (lane >= m) incl += y;
    }
    const int k = p - (int)wave_sum((uint32_t)mine);
    const unsigned long long reach = __ballot((int)incl > k);
    if (!reach) return u;
    u.n = __builtin_ctzll(reach);
    u.column = __shfl(mine + k - (int)(incl - at), u.n, 64);
    return u;
}

// x as the sum of TERMS bf16 values.
template <int TERMS> __device__ __forceinline__ void terms_of(float x, int e, bf16x8 (&t)[TERMS]) {
#pragma unroll
    for (int i = 0; i < TERMS; ++i) {
        const __bf16 y = (__bf16)x;
        t[i][e] = y;
        if (i + 1 < TERMS) x -= (float)y;
    }
}

// Eight e4m3 values (two words) as bf16, times a power of two.
__device__ __forceinline__ bf16x8 widen(uint32_t lo, uint32_t hi, float scale) {
    const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, scale, false), b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, scale, true);
    const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, scale, false), d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, scale, true);
    return bf16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

__device__ __forceinline__ f32x4 mma(bf16x8 a, bf16x8 b, f32x4 c) { return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0); }

// Bytes of w that are NaN, as 0x80 in each.
__device__ __forceinline__ uint32_t nan_bytes(uint32_t w) { return ((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u; }

// Max over the four lane groups, in every lane.
__device__ __forceinline__ float group_max(float x) {
    const uint32_t b = __float_as_uint(x);
    const auto p = __builtin_amdgcn_permlane16_swap(b, b, false, false);
    x = __builtin_fmaxf(__uint_as_float(p[0]), __uint_as_float(p[1]));
    const uint32_t c = __float_as_uint(x);
    const auto q = __builtin_amdgcn_permlane32_swap(c, c, false, false);
    return __builtin_fmaxf(__uint_as_float(q[0]), __uint_as_float(q[1]));
}

// A load of what is read once in a launch (ONCE), or again by other workgroups.
template <bool ONCE, typename W> __device__ __forceinline__ W once(const W *p) {
    if constexpr (ONCE) return __builtin_nontemporal_load(p);
    else return *p;
}

template <int N> struct Bytes;   // of one lane's share of a row of values
template <> struct Bytes<16> { u32x4 w; };
template <> struct Bytes<8> { u32x2 w; };

// KEYS keys a step.  64 take 16 bytes a lane of keys and of values; 32 leave room
// for twice the columns in the registers of two waves a SIMD, whose matrix and
// vector instructions then overlap, with the queries in LDS.
template <typename T, int D, int NT, int KEYS, bool SPLIT>
__global__ __launch_bounds__(kThreads, sizeof(T) == 4 && !SPLIT ? 1 : 2) void attend_kernel(const AttendArgs a, const Plan plan) {
    constexpr int TERMS = sizeof(T) == 4 ? 3 : 1, KL = D / 64, MT = D / 16, WAVE = 16 * NT, COLS = SPLIT ? WAVE : kWaves * WAVE;
    constexpr int PTERMS = TERMS == 1 && SPLIT ? 2 : TERMS;         // of a numerator
    constexpr int ST = KEYS / 16, PS = KEYS / 32, OWN = KEYS / 4;   // score tiles, product steps, keys of a lane group
    constexpr bool QLDS = !SPLIT;
    constexpr int QBYTES = QLDS ? kWaves * NT * KL * 2 * TERMS * 1024 : 16, JOIN = kWaves * 4 * 256 * 4;
    __shared__ __align__(16) unsigned char pool[QBYTES > JOIN ? QBYTES : JOIN];   // the queries, then the waves' sums
    __shared__ float stats[kWaves][WAVE][2];
    float (*joined)[4][256] = reinterpret_cast<float (*)[4][256]>(pool);
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, c = lane & 15, grp = lane >> 4;
    const int head = blockIdx.x % a.heads, place = blockIdx.x / a.heads, g = a.q_heads / a.heads;
    const Unit u = plan.starts ? planned_unit_of(a, plan, place, g, COLS, KEYS)
                   : !SPLIT && plan.places == plan.units && a.num_seqs <= 64 ? longest_unit_of(a, place, g, COLS, KEYS)
                                                                             : unit_of(a, plan, place, g, COLS, KEYS);
    if (u.n < 0) return;
    const Request r = request_of(a, u.n, g, COLS, KEYS);
    // the last columns first: they see the most keys
    const int all = r.length * g, first = (r.units - 1 - u.column) * COLS, end = min(first + COLS, all);
    const int before = r.total - r.length;                                // position of the request's first token
    const int unit_keys = max(before + (end - 1) / g + 1, 0);
    const int unit_tiles = (unit_keys + KEYS - 1) / KEYS;
    const int chunks = max(1, (unit_tiles + u.length - 1) / u.length);    // that this unit really has
    if (u.chunk >= chunks) return;
    if (plan.places > plan.units && u.chunk == 0)                         // for the launch that joins the chunks
        for (int col = first + threadIdx.x; col < end; col += kThreads) {
            const int token = col / g;
            int *to = plan.info + 2 * ((long)(r.begin + token) * a.q_heads + (long)head * g + (col - token * g));
            to[0] = place;
            to[1] = chunks << 8 | (col - first);
        }
    const bool same = SPLIT || end - first <= WAVE;                       // the waves share columns and split the keys
    const int col0 = first + (same ? 0 : wave * WAVE), col1 = min(col0 + WAVE, end);
    const int seen = col1 > col0 ? max(before + (col1 - 1) / g + 1, 0) : 0;   // keys that some column of this wave sees
    const int least = col1 > col0 ? before + col0 / g : -1;                   // the last key that all of them see
    const int step = same ? kWaves : 1;
    const int stop = min((u.chunk + 1) * u.length, (seen + KEYS - 1) / KEYS);
    int tile = u.chunk * u.length + (same ? wave : 0);

    // queries
    bf16x8 qreg[QLDS ? 1 : NT][KL][2][TERMS];
    bf16x8 *qlds = reinterpret_cast<bf16x8 *>(pool) + wave * (NT * KL * 2 * TERMS * 64) + lane;
    const auto query = [&](int nt, int j, int h, int i) {
        if constexpr (QLDS) return qlds[(((nt * KL + j) * 2 + h) * TERMS + i) * 64];
        else return qreg[nt][j][h][i];
    };
    int last[NT];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        const int col = col0 + 16 * nt + c;
        const bool in = col < col1;
        const int token = in ? col / g : 0, h = in ? col - token * g : 0;
        last[nt] = in ? before + token : -1;
        const T *src = static_cast<const T *>(a.q) + (long)(r.begin + token) * a.q_stride + ((long)head * g + h) * D;
#pragma unroll
        for (int j = 0; j < KL; ++j)
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const T *at = src + 64 * j + 16 * grp + 8 * s;
                bf16x8 t[TERMS];
                if constexpr (TERMS == 1) {
                    u32x4 w{0, 0, 0, 0};
                    if (in) w = *reinterpret_cast<const u32x4 *>(at);
                    t[0] = __builtin_bit_cast(bf16x8, w);
                } else {
                    f32x4 x{0.f, 0.f, 0.f, 0.f}, y{0.f, 0.f, 0.f, 0.f};
                    if (in) {
                        x = load4(at);
                        y = load4(at + 4);
                    }
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        terms_of<TERMS>(x[e], e, t);
                        terms_of<TERMS>(y[e], 4 + e, t);
                    }
                }
#pragma unroll
                for (int i = 0; i < TERMS; ++i) {
                    if constexpr (QLDS) qlds[(((nt * KL + j) * 2 + s) * TERMS + i) * 64] = t[i];
                    else qreg[nt][j][s][i] = t[i];
                }
            }
    }

    const int bs = 1 << a.block_shift, within = bs - 1;
    const int32_t *table = a.block_table + (long)a.indices[u.n] * a.max_blocks;
    const float to2 = a.scale * kLog2e;
    const auto page = [&](int tile, int group) {
        const int i = (tile * KEYS + OWN * group) >> a.block_shift;
        return table[min(i, a.max_blocks - 1)];
    };
    u32x4 kr[ST][KL];
    Bytes<OWN> vr[MT];
    float ks, vs;
    bool fine;   // this lane's keys begin in a block that holds some
    const auto load_k = [&](int tile, int block) {
        const int b = (unsigned)block < (unsigned)a.num_blocks ? block : 0, off = (tile * KEYS + OWN * (c >> 2)) & within;
        const long at = (long)b * a.heads + head;
        ks = a.k_scale[at];
        const uint8_t *p = a.k_cache + (at * bs + off + (c & 3)) * D + 16 * grp;
#pragma unroll
        for (int t = 0; t < ST; ++t)
#pragma unroll
            for (int j = 0; j < KL; ++j) kr[t][j] = once<SPLIT>(reinterpret_cast<const u32x4 *>(p + 4 * t * D + 64 * j));
    };
    const auto load_v = [&](int tile, int block) {
        fine = (unsigned)block < (unsigned)a.num_blocks && tile * KEYS + OWN * grp < r.total;
        const int b = fine ? block : 0, off = (tile * KEYS + OWN * grp) & within;
        const long at = (long)b * a.heads + head;
        vs = fine ? a.v_scale[at] : 1.f;
        const uint8_t *p = a.v_cache + (at * D + c) * bs + off;
#pragma unroll
        for (int t = 0; t < MT; ++t) vr[t].w = once<SPLIT>(reinterpret_cast<const decltype(Bytes<OWN>::w) *>(p + 16 * t * bs));
    };

    f32x4 o[MT][NT];
    float m[NT], l[NT];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        m[nt] = kNone;
        l[nt] = 0.f;
#pragma unroll
        for (int t = 0; t < MT; ++t) o[t][nt] = f32x4{0.f, 0.f, 0.f, 0.f};
    }

    if (tile < stop) {
        load_k(tile, page(tile, c >> 2));
        load_v(tile, page(tile, grp));
    }
    for (; tile < stop; tile += step) {
        const int next = min(tile + step, stop - 1);   // the last one is loaded again, unused
        const int kpage = page(next, c >> 2), vpage = page(next, grp);
        f32x4 s[ST][NT];
#pragma unroll
        for (int t = 0; t < ST; ++t)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) s[t][nt] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int j = 0; j < KL; ++j)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                bf16x8 k[ST];
#pragma unroll
                for (int t = 0; t < ST; ++t) k[t] = widen(kr[t][j][2 * h], kr[t][j][2 * h + 1], ks);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int i = TERMS - 1; i >= 0; --i) {
                        const bf16x8 q = query(nt, j, h, i);
#pragma unroll
                        for (int t = 0; t < ST; ++t) s[t][nt] = mma(k[t], q, s[t][nt]);
                    }
            }
        load_k(next, kpage);
        const bool masked = tile * KEYS + KEYS - 1 > least || __any(!fine);
        if (masked) {
            asm volatile("");   // a branch: most tiles have nothing to hide
#pragma unroll
            for (int t = 0; t < ST; ++t)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (!fine || tile * KEYS + OWN * grp + 4 * t + i > last[nt]) s[t][nt][i] = -__builtin_inff();
        }
        // A reference that holds until a score passes it by 2^8; whether one does is
        // asked of every lane's own scores, and the column's largest sought only then.
        float top[NT];
        bool raise = false;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            float x = s[0][nt][0];
#pragma unroll
            for (int t = 0; t < ST; ++t)
#pragma unroll
                for (int i = 0; i < 4; ++i) x = __builtin_fmaxf(x, s[t][nt][i]);
            top[nt] = x;
            raise |= (x - m[nt]) * to2 > 8.f;
        }
        if (__any(raise)) {
            asm volatile("");
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const float to = __builtin_fmaxf(m[nt], group_max(top[nt])), f = __builtin_amdgcn_exp2f((m[nt] - to) * to2);
                m[nt] = to;
                l[nt] *= f;
#pragma unroll
                for (int t = 0; t < MT; ++t)
#pragma unroll
                    for (int i = 0; i < 4; ++i) o[t][nt][i] *= f;
            }
        }
        bf16x8 p[NT][PS];   // the numerators, where one term is all of them; more are formed where they are used
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const float shift = -m[nt] * to2;
#pragma unroll
            for (int t = 0; t < ST; ++t)
#pragma unroll
                for (int i = 0; i < 4; i += 2) {
                    const float x = __builtin_amdgcn_exp2f(__builtin_fmaf(s[t][nt][i], to2, shift));
                    const float y = __builtin_amdgcn_exp2f(__builtin_fmaf(s[t][nt][i + 1], to2, shift));
                    if constexpr (PTERMS == 1) {   // the sum of what the product sees, two at a time
                        const bf16x2 z{(__bf16)x, (__bf16)y};
                        p[nt][t >> 1][4 * (t & 1) + i] = z[0];
                        p[nt][t >> 1][4 * (t & 1) + i + 1] = z[1];
                        l[nt] = __builtin_amdgcn_fdot2_f32_bf16(z, bf16x2{(__bf16)1.f, (__bf16)1.f}, l[nt], false);
                    } else {
                        l[nt] += x;
                        l[nt] += y;
                        s[t][nt][i] = x;
                        s[t][nt][i + 1] = y;
                    }
                }
        }
        if (masked) {
            asm volatile("");
            // what a column must not see may be NaN, and 0 * NaN would reach it
            uint32_t bad = 0;
#pragma unroll
            for (int t = 0; t < MT; ++t)
#pragma unroll
                for (int i = 0; i < OWN / 4; ++i) bad |= nan_bytes(vr[t].w[i]);
            if (__any(bad != 0)) {
                asm volatile("");
                // the NaN among the values become zeros here, and NaN in the columns that see them
#pragma unroll 1
                for (int h = 0; h < PS; ++h) {
                    bf16x8 one[NT];
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            one[nt][e] = (__bf16)(!fine || tile * KEYS + OWN * grp + 8 * h + e > last[nt] ? 0.f : 1.f);
#pragma unroll
                    for (int t = 0; t < MT; ++t) {
                        uint32_t flag[2];
#pragma unroll
                        for (int i = 0; i < 2; ++i) flag[i] = (nan_bytes(PS == 1 || h == 0 ? vr[t].w[i] : vr[t].w[OWN / 4 - 2 + i]) >> 7) * 0x38u;   // e4m3's one
                        const bf16x8 f = widen(flag[0], flag[1], 1.f);
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            const f32x4 hit = mma(f, one[nt], f32x4{0.f, 0.f, 0.f, 0.f});
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                if (hit[i] > 0.f) o[t][nt][i] = __builtin_nanf("");
                        }
                    }
                }
#pragma unroll
                for (int t = 0; t < MT; ++t)
#pragma unroll
                    for (int i = 0; i < OWN / 4; ++i) vr[t].w[i] &= ~((nan_bytes(vr[t].w[i]) >> 7) * 0xffu);
            }
        }
        if constexpr (PTERMS == 1) {
#pragma unroll
            for (int t = 0; t < MT; ++t)
#pragma unroll
                for (int h = 0; h < PS; ++h) {
                    const bf16x8 v = widen(vr[t].w[2 * h], vr[t].w[2 * h + 1], vs);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) o[t][nt] = mma(v, p[nt][h], o[t][nt]);
                }
        } else {
#pragma unroll
            for (int h = 0; h < PS; ++h) {
                bf16x8 z[NT][PTERMS];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 8; ++e) terms_of<PTERMS>(s[2 * h + e / 4][nt][e % 4], e, z[nt]);
#pragma unroll
                for (int t = 0; t < MT; ++t) {
                    const bf16x8 v = widen(vr[t].w[2 * h], vr[t].w[2 * h + 1], vs);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int i = PTERMS - 1; i >= 0; --i) o[t][nt] = mma(v, z[nt][i], o[t][nt]);
                }
            }
        }
        load_v(next, vpage);
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        l[nt] += __shfl_xor(l[nt], 16, 64);
        l[nt] += __shfl_xor(l[nt], 32, 64);
    }

    const bool alone = chunks == 1;
    const long at = (long)place * a.heads + head;
    // channels 16 t + 4 grp .. + 3 of column c of tile nt
    const auto write = [&](int t, int nt, int col, f32x4 x, float sum) {
        if (col >= end) return;
        const int d = 16 * t + 4 * grp;
        if (alone) {
            const int token = col / g, h = col - token * g;
            T *to = static_cast<T *>(a.o) + ((long)(r.begin + token) * a.q_heads + (long)head * g + h) * D + d;
            const float f = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
            for (int i = 0; i < 4; ++i) x[i] *= f;
            if constexpr (sizeof(T) == 4) *reinterpret_cast<f32x4 *>(to) = x;
            else *reinterpret_cast<u32x2 *>(to) = u32x2{pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3])};
        } else {
            *reinterpret_cast<f32x4 *>(plan.parts + (at * COLS + col - first) * D + d) = x;
        }
    };
    if (!same) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int col = col0 + 16 * nt + c;
#pragma unroll
            for (int t = 0; t < MT; ++t) write(t, nt, col, o[t][nt], l[nt]);
            if (!alone && grp == 0 && col < end) *reinterpret_cast<f32x2 *>(plan.sums + (at * COLS + col - first) * 2) = f32x2{m[nt], l[nt]};
        }
        return;
    }
    // the waves' sums come together
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
        if (grp == 0) {
            stats[wave][16 * nt + c][0] = m[nt];
            stats[wave][16 * nt + c][1] = l[nt];
        }
    __syncthreads();   // and no wave needs its queries any more
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        float to = kNone, sum = 0.f;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) to = __builtin_fmaxf(to, stats[w][16 * nt + c][0]);
#pragma unroll
        for (int w = 0; w < kWaves; ++w) sum += stats[w][16 * nt + c][1] * __builtin_amdgcn_exp2f((stats[w][16 * nt + c][0] - to) * to2);
        const float f = __builtin_amdgcn_exp2f((m[nt] - to) * to2);
        const int col = col0 + 16 * nt + c;
#pragma unroll
        for (int t0 = 0; t0 < MT; t0 += 4) {
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                f32x4 x = o[t0 + t][nt];
#pragma unroll
                for (int i = 0; i < 4; ++i) x[i] *= f;
                *reinterpret_cast<f32x4 *>(&joined[wave][t][4 * lane]) = x;
            }
            __syncthreads();
            f32x4 x = *reinterpret_cast<const f32x4 *>(&joined[0][wave][4 * lane]);
#pragma unroll
            for (int w = 1; w < kWaves; ++w) x += *reinterpret_cast<const f32x4 *>(&joined[w][wave][4 * lane]);
            write(t0 + wave, nt, col, x, sum);
            __syncthreads();
        }
        if (!alone && wave == 0 && grp == 0 && col < end) *reinterpret_cast<f32x2 *>(plan.sums + (at * COLS + col - first) * 2) = f32x2{to, sum};
    }
}

// The chunks of a column (token, query head) joined; one wave a column.
template <typename T, int D> __global__ __launch_bounds__(256) void join_kernel(const AttendArgs a, const Plan plan, int cols) {
    const int lane = threadIdx.x & 63;
    const long column = (long)blockIdx.x * 4 + (threadIdx.x >> 6);
    const int token = (int)(column / a.q_heads), head = (int)(column % a.q_heads) / (a.q_heads / a.heads);
    if (token >= min(a.cu_seqlens[a.num_seqs], a.total_tokens)) return;
    const uint32_t place = (uint32_t)plan.info[2 * column], chunks = (uint32_t)plan.info[2 * column + 1] >> 8;
    const int col = plan.info[2 * column + 1] & 0xff;
    if (chunks == 1 || (long)place + chunks > plan.places) return;   // (never more than there are, if the offsets fit the call)
    const float to2 = a.scale * kLog2e;
    const auto at = [&](int k) { return ((long)(place + k) * a.heads + head) * cols + col; };
    float top = kNone, sum = 0.f, x[D / 64];
#pragma unroll
    for (int i = 0; i < D / 64; ++i) x[i] = 0.f;
    for (int k0 = 0; k0 < (int)chunks; k0 += 64) {   // a chunk a lane
        const int some = min((int)chunks - k0, 64);
        f32x2 ml{kNone, 0.f};
        if (lane < some) ml = *reinterpret_cast<const f32x2 *>(plan.sums + at(k0 + lane) * 2);
        float m = ml[0];
#pragma unroll
        for (int d = 32; d >= 1; d >>= 1) m = __builtin_fmaxf(m, __shfl_xor(m, d, 64));
        const float next = __builtin_fmaxf(top, m), f = __builtin_amdgcn_exp2f((ml[0] - next) * to2), again = __builtin_amdgcn_exp2f((top - next) * to2);
        top = next;
        sum = sum * again + group_sum<64>(f * ml[1]);
#pragma unroll
        for (int i = 0; i < D / 64; ++i) x[i] *= again;
        constexpr int AHEAD = 8;
        for (int k = 0; k < some; k += AHEAD) {
            float y[AHEAD][D / 64];
#pragma unroll
            for (int e = 0; e < AHEAD; ++e)
#pragma unroll
                for (int i = 0; i < D / 64; ++i) y[e][i] = plan.parts[at(k0 + min(k + e, some - 1)) * D + lane + 64 * i];
#pragma unroll
            for (int e = 0; e < AHEAD; ++e) {
                const float g = __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(f), min(k + e, 63)));
#pragma unroll
                for (int i = 0; i < D / 64; ++i)
                    if (k + e < some) x[i] += g * y[e][i];
            }
        }
    }
    T *to = static_cast<T *>(a.o) + column * D;
    const float f = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
    for (int i = 0; i < D / 64; ++i) io_traits<T>::store(to, lane + 64 * i, x[i] * f);
}

template <typename T, int D, int NT, int KEYS, bool SPLIT>
hipError_t launch(const AttendArgs &a, const Layout &y, const Plan &plan, hipStream_t stream) {
    if (plan.starts) plan_kernel<<<1, kPlanThreads, 0, stream>>>(a, plan, y.cols, KEYS);
    attend_kernel<T, D, NT, KEYS, SPLIT><<<(unsigned)(plan.places * a.heads), kThreads, 0, stream>>>(a, plan);
    if (plan.places > plan.units) {
        const long columns = (long)a.total_tokens * a.q_heads;
        join_kernel<T, D><<<(unsigned)((columns + 3) / 4), 256, 0, stream>>>(a, plan, y.cols);
    }
    return hipGetLastError();
}

template <typename T, int D> hipError_t launch(const AttendArgs &a, const Layout &y, const Plan &plan, hipStream_t stream) {
    if (y.split) return y.nt == 1 ? launch<T, D, 1, 64, true>(a, y, plan, stream) : launch<T, D, 2, 64, true>(a, y, plan, stream);
    if constexpr (sizeof(T) == 4) return launch<T, D, 2, 32, false>(a, y, plan, stream);
    else return launch<T, D, 4, 32, false>(a, y, plan, stream);
}

}  // namespace

size_t attend_workspace_bytes(int num_seqs, int total_tokens, int q_heads, int heads, int d, bool io_bf16) {
    const Layout y = layout_of(num_seqs, total_tokens, q_heads, heads, io_bf16);
    if (y.places == y.units) return starts_bytes(num_seqs);
    return starts_bytes(num_seqs) + info_bytes((long)total_tokens * q_heads) + (size_t)y.places * heads * y.cols * (d + 2) * sizeof(float);
}

long attend_grid(int num_seqs, int total_tokens, int q_heads, int heads, int d, bool io_bf16) {
    const Layout y = layout_of(num_seqs, total_tokens, q_heads, heads, io_bf16);
    return std::max(y.places * heads, ((long)total_tokens * q_heads + 3) / 4);
}

hipError_t launch_attend(const AttendArgs &a, void *workspace, hipStream_t stream) {
    const Layout y = layout_of(a.num_seqs, a.total_tokens, a.q_heads, a.heads, a.io_bf16);
    Plan plan{};
    plan.units = (int)y.units;
    plan.places = (int)y.places;
    // Tiles of a chunk at least.  Single tokens: two for each of the four waves (one
    // request of 8000 tokens 14 us, with one 20).  Prompts: a chunk's sums of all its
    // columns are written and read once more, 128 KB for 256 columns of 128 channels, so
    // 512 keys (6 prompts of up to 409 tokens, 200 workgroups: 28 us, with 128 keys 46),
    // but 128 where the undivided columns are no 96 workgroups (one of 1889 tokens over
    // 2 heads, 30 workgroups: 21 us, with 512 keys 27).
    plan.least = y.split ? 8 : y.units * a.heads < 96 ? 4 : a.io_bf16 ? 16 : 8;
    char *at = static_cast<char *>(workspace);
    if (starts_bytes(a.num_seqs)) plan.starts = reinterpret_cast<uint32_t *>(at);
    at += starts_bytes(a.num_seqs);
    plan.info = reinterpret_cast<int *>(at);
    plan.parts = reinterpret_cast<float *>(at + info_bytes((long)a.total_tokens * a.q_heads));
    plan.sums = plan.parts + (size_t)y.places * a.heads * y.cols * a.d;
    if (a.io_bf16) return a.d == 64 ? launch<bf16, 64>(a, y, plan, stream) : launch<bf16, 128>(a, y, plan, stream);
    return a.d == 64 ? launch<float, 64>(a, y, plan, stream) : launch<float, 128>(a, y, plan, stream);
}

}  // namespace kda
