// Verification of drafted tokens against the target's probabilities, and the
// commit of the accepted states.
//
// A request's drafts are tested 64 at a time, one a lane; the first refused
// one gives the row whose rest the next token is drawn from.  That row (and
// the drafts' own, where one was refused) is read once, in parts of a few
// thousand tokens summed by a wave in fp64; the part that holds r times the
// total is found from the sums, and only that part is read again to find the
// token.  Bound by those rows' bytes with many requests, by the chain of
// dependent loads with one.  Measured: 1024 requests with rows of 65,536 (fp32,
// runs of four, 0.43 GB) 88 us, 4.9 TB/s; one request, 131,072 tokens: 11 us
// (4.9 the sums, 3.6 the token, two launches).
#include "kda_device.h"
#include "kda_internal.h"

namespace kda {

constexpr int kVerifyWaves = 8;
constexpr int kVerifyThreads = kVerifyWaves * 64;
constexpr int kVerifyParts = 256;                  // most parts of a row
constexpr int kVec = 4;                            // neighbouring tokens of a lane
constexpr int kPart = 4 * 64 * kVec;               // tokens of a part: a multiple of this

static int part_tokens(int vocab) {
    return (int)((((long)vocab + kVerifyParts - 1) / kVerifyParts + kPart - 1) / kPart * kPart);
}
int verify_parts(int vocab) { return (int)(((long)vocab + part_tokens(vocab) - 1) / part_tokens(vocab)); }

// Workgroups a row's parts are summed by.  One finds the token as well, in one
// launch; with more a wave takes a part and a second launch finds the token.
// One is for rows of 8 waves' parts, and for many requests with rows of up to
// 32 parts.  Measured with runs of four, one against several (us):
//     tokens    1 request      128          256         512         1024
//     32,768    22 / 14     25 / 21     32 / 38     49 / 51     84 / 84
//     65,536    32 / 14     42 / 33     50 / 51     82 / 81    138 / 135
//     131,072   54 / 13     72 / 50     87 / 80    134 / 127   218 / 198
static int verify_groups(int num_seqs, int parts) {
    return num_seqs >= 256 && parts <= 32 ? 1 : (parts + kVerifyWaves - 1) / kVerifyWaves;
}

struct Verdict {
    int t0, len, accepted;   // accepted: drafts that stood
    int wrong;               // the refused draft, or -1 where every one stood
    bool refused;
};

template <typename PT> __device__ __forceinline__ Verdict verdict_of(const VerifyArgs &a, int n, int lane) {
    Verdict v;
    v.t0 = a.cu_seqlens[n];
    v.len = a.cu_seqlens[n + 1] - v.t0;
    v.accepted = v.len - 1;
    v.wrong = -1;
    for (int base = 0; base < v.len - 1; base += 64) {
        const int j = base + lane;
        bool bad = false;
        int d = -1;
        if (j < v.len - 1) {
            const long t = v.t0 + j;
            d = a.tokens[t + 1];
            bad = true;
            if (d >= 0 && d < a.vocab) {
                const float p = io_traits<PT>::load(reinterpret_cast<const PT *>(a.target) + t * a.target_stride, d);
                const float q = a.draft ? io_traits<PT>::load(reinterpret_cast<const PT *>(a.draft) + t * a.draft_stride, d) : 1.f;
                bad = !(a.uniform[t] * q < p);
            }
        }
        const unsigned long long m = __ballot(bad);
        if (m) {
            const int first = __builtin_ctzll(m);
            v.accepted = base + first;
            v.wrong = __shfl(d, first, 64);
            break;
        }
    }
    v.refused = v.accepted < v.len - 1;
    return v;
}

// The refused (or last) row: weights w and p's own.
template <typename PT> struct Row {
    const PT *p, *q;   // q: NULL where nothing is taken off
    int wrong;         // token of weight 0, or -1
    int vocab;
    bool wide;         // rows start on 16 (bf16: 8) bytes

    // Tokens i .. i + 3; those past the vocabulary weigh nothing.
    __device__ __forceinline__ void at(int i, float (&w)[kVec], float (&own)[kVec]) const {
        f32x4 x = {0.f, 0.f, 0.f, 0.f}, y = x;
        if (wide && i + kVec <= vocab) {
            x = load4(p + i);
            if (q) y = load4(q + i);
        } else {
#pragma unroll
            for (int e = 0; e < kVec; ++e)
                if (i + e < vocab) {
                    x[e] = io_traits<PT>::load(p, i + e);
                    if (q) y[e] = io_traits<PT>::load(q, i + e);
                }
        }
#pragma unroll
        for (int e = 0; e < kVec; ++e) {
            own[e] = fmaxf(x[e], 0.f);   // NaN weighs nothing
            w[e] = q ? fmaxf(x[e] - y[e], 0.f) : i + e == wrong ? 0.f : own[e];
        }
    }
};

template <typename PT> __device__ __forceinline__ Row<PT> row_of(const VerifyArgs &a, const Verdict &v) {
    const long t = v.t0 + v.accepted;
    Row<PT> r;
    r.p = reinterpret_cast<const PT *>(a.target) + t * a.target_stride;
    r.q = a.draft && v.refused ? reinterpret_cast<const PT *>(a.draft) + t * a.draft_stride : nullptr;
    r.wrong = v.refused ? v.wrong : -1;
    r.vocab = a.vocab;
    r.wide = a.target_stride % kVec == 0 && a.draft_stride % kVec == 0;
    return r;
}

// A wave's sums of one part: of the weights and of p.
template <typename PT>
__device__ __forceinline__ void sum_part(const Row<PT> &r, int lo, int hi, int lane, double &w, double &own) {
    w = 0.0;
    own = 0.0;
    for (int base = lo; base < hi; base += kPart) {
#pragma unroll
        for (int k = 0; k < kPart / (64 * kVec); ++k) {
            float x[kVec], o[kVec];
            r.at(base + (k * 64 + lane) * kVec, x, o);
#pragma unroll
            for (int e = 0; e < kVec; ++e) {
                w += (double)x[e];
                own += (double)o[e];
            }
        }
    }
    w = lane_value(wave_scan(w), 63);
    own = lane_value(wave_scan(own), 63);
}

// The part of a row that holds `want` = r times the total, from the sums of
// all parts (every wave finds the same): its number, or -1 where no part has
// any weight, and the sum before it.
__device__ __forceinline__ int find_part(const double *sums, int parts, float r, int lane, double &want, double &before) {
    constexpr int EACH = kVerifyParts / 64;
    double s[EACH], own = 0.0;
#pragma unroll
    for (int k = 0; k < EACH; ++k) {
        const int i = lane * EACH + k;
        s[k] = i < parts ? sums[i] : 0.0;
        own += s[k];
    }
    const double cum = wave_scan(own), total = lane_value(cum, 63);
    want = (double)r * total;
    double c = cum - own, at = 0.0;
    int hit = -1, last = -1;   // first part past `want`; the last with any weight where rounding (or r = 1) leaves none
#pragma unroll
    for (int k = 0; k < EACH; ++k) {
        if (s[k] > 0.0) {
            last = lane * EACH + k;
            if (hit < 0) {
                at = c;
                if (c + s[k] > want) hit = last;
            }
        }
        c += s[k];
    }
    const unsigned long long past = __ballot(hit >= 0), some = __ballot(last >= 0);
    if (!some) return -1;
    const int from = past ? __builtin_ctzll(past) : 63 - __builtin_clzll(some);
    before = lane_value(at, from);
    return __builtin_amdgcn_readlane(past ? hit : last, from);
}

// The whole workgroup: finds the token and writes the request's outputs.
// sums: of the weights of all parts, then of p of all parts.
template <typename PT>
__device__ void pick(const VerifyArgs &a, int n, const Verdict &v, const Row<PT> &r, const double *sums, int part_len) {
    __shared__ double totals[kVerifyWaves];
    __shared__ int hits[kVerifyWaves], lasts[kVerifyWaves];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    double want = 0.0, carry = 0.0;
    bool rest = true;
    int part = find_part(sums, a.parts, a.uniform_next[n], lane, want, carry), next = -1;
    if (part < 0) {   // nothing is left of the row: p itself
        rest = false;
        part = find_part(sums + a.parts, a.parts, a.uniform_next[n], lane, want, carry);
    }
    if (part >= 0) {
        const int lo = part * part_len, hi = (int)min((long)a.vocab, (long)lo + part_len);
        for (int base = lo; base < hi; base += kVerifyThreads * kVec) {
            const int i = base + tid * kVec;
            float x[kVec], o[kVec];
            r.at(i, x, o);
            double own = 0.0;
#pragma unroll
            for (int e = 0; e < kVec; ++e) {
                x[e] = i + e >= hi ? 0.f : rest ? x[e] : o[e];
                own += (double)x[e];
            }
            const double cum = wave_scan(own);
            if (lane == 63) totals[wave] = cum;
            __syncthreads();
            double c = carry + (cum - own);
#pragma unroll
            for (int k = 0; k < kVerifyWaves; ++k) {
                if (k < wave) c += totals[k];
                carry += totals[k];
            }
            // the first token past `want`; failing that the last with any weight
            int hit = -1, last = -1;
#pragma unroll
            for (int e = 0; e < kVec; ++e) {
                c += (double)x[e];
                if (x[e] > 0.f) {
                    last = i + e;
                    if (hit < 0 && c > want) hit = i + e;
                }
            }
            const unsigned long long past = __ballot(hit >= 0), some = __ballot(last >= 0);
            hit = past ? __builtin_amdgcn_readlane(hit, __builtin_ctzll(past)) : -1;
            last = some ? __builtin_amdgcn_readlane(last, 63 - __builtin_clzll(some)) : -1;
            if (lane == 0) {
                hits[wave] = hit;
                lasts[wave] = last;
            }
            __syncthreads();
            hit = -1;
#pragma unroll
            for (int k = 0; k < kVerifyWaves; ++k) {
                if (hit < 0) hit = hits[k];
                if (lasts[k] >= 0) last = lasts[k];
            }
            if (hit >= 0 || last >= 0) next = hit >= 0 ? hit : last;
            __syncthreads();   // before the next tokens' totals and hits
            if (hit >= 0) break;
        }
    }
    if (tid == 0) {
        a.accepted[n] = v.accepted;
        a.next[n] = next;
    }
    for (int j = tid; j < v.len; j += kVerifyThreads)
        a.emitted[v.t0 + j] = j < v.accepted ? a.tokens[v.t0 + j + 1] : j == v.accepted ? next : -1;
}

// What the first launch leaves for the second: [N] verdicts, then the sums.
struct Left { int accepted, wrong; };

// grid (workgroups of a row, requests on y and z): sums the parts; with one
// workgroup a row also finds the token.
template <typename PT> __global__ __launch_bounds__(kVerifyThreads) void verify_sum_kernel(VerifyArgs a, int part_len) {
    __shared__ double sums[2 * kVerifyParts];
    const int n = (int)blockIdx.y + (int)blockIdx.z * (int)gridDim.y;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    if (n >= a.num_seqs) return;
    const Verdict v = verdict_of<PT>(a, n, lane);
    if (v.len <= 0) {
        if (blockIdx.x == 0 && threadIdx.x == 0) {
            a.accepted[n] = -1;
            a.next[n] = -1;
        }
        return;
    }
    const bool alone = gridDim.x == 1;
    double *out = alone ? sums : a.partial + a.num_seqs + (long)n * 2 * a.parts;
    if (!alone && blockIdx.x == 0 && threadIdx.x == 0) reinterpret_cast<Left *>(a.partial)[n] = Left{v.accepted, v.wrong};
    const Row<PT> r = row_of<PT>(a, v);
    for (int part = (int)blockIdx.x * kVerifyWaves + wave; part < a.parts; part += (int)gridDim.x * kVerifyWaves) {
        double w, own;
        const int lo = part * part_len;
        sum_part<PT>(r, lo, (int)min((long)a.vocab, (long)lo + part_len), lane, w, own);
        if (lane == 0) {
            out[part] = w;
            out[a.parts + part] = own;
        }
    }
    if (!alone) return;
    __syncthreads();
    pick<PT>(a, n, v, r, sums, part_len);
}

// grid (1, requests on y and z): the token from the parts' sums.
template <typename PT> __global__ __launch_bounds__(kVerifyThreads) void verify_pick_kernel(VerifyArgs a, int part_len) {
    const int n = (int)blockIdx.y + (int)blockIdx.z * (int)gridDim.y;
    if (n >= a.num_seqs) return;
    Verdict v;
    v.t0 = a.cu_seqlens[n];
    v.len = a.cu_seqlens[n + 1] - v.t0;
    if (v.len <= 0) return;
    const Left left = reinterpret_cast<const Left *>(a.partial)[n];
    v.accepted = left.accepted;
    v.wrong = left.wrong;
    v.refused = v.accepted < v.len - 1;
    pick<PT>(a, n, v, row_of<PT>(a, v), a.partial + a.num_seqs + (long)n * 2 * a.parts, part_len);
}

template <typename PT> static hipError_t launch_p(const VerifyArgs &a, hipStream_t s) {
    const dim3 grid(verify_groups(a.num_seqs, a.parts), decode_grid_y(a.num_seqs), decode_grid_z(a.num_seqs));
    const int part_len = part_tokens(a.vocab);
    verify_sum_kernel<PT><<<grid, kVerifyThreads, 0, s>>>(a, part_len);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || grid.x == 1) return e;
    verify_pick_kernel<PT><<<dim3(1, grid.y, grid.z), kVerifyThreads, 0, s>>>(a, part_len);
    return hipGetLastError();
}
hipError_t launch_verify(const VerifyArgs &a, hipStream_t s) { return a.bf16 ? launch_p<bf16>(a, s) : launch_p<float>(a, s); }

// ---- commit ----------------------------------------------------------------

// Rows are copied through buffer resources, eight 16-byte accesses a thread
// back to back with no branch between them (the range check ends a row):
// 1024 states of 1 MB with their convolutions' inputs 522 -> 407 us, 5.4 TB/s.
// Both sides pass the caches by (nt): 407 us with it, 426 without, 408 with
// device scope (sc1) as well.
constexpr int kCommitLoads = 8, kCommitBytes = 256 * 16 * kCommitLoads, kPassCaches = 2;

// grid (blocks of a row, requests on y and z)
__global__ __launch_bounds__(256) void commit_kernel(const int32_t *indices, const int32_t *steps, const char *cache, char *pool,
                                                     int num_seqs, int num_slots, int cache_steps, int cache_pitch,
                                                     long row_bytes) {
    const int n = (int)blockIdx.y + (int)blockIdx.z * (int)gridDim.y;
    if (n >= num_seqs) return;
    const int step = steps[n];
    if (step < 0 || step >= cache_steps) return;
    long slot = indices[n];
    if (slot < 0) slot = num_slots - 1;
    const long at = (long)blockIdx.x * kCommitBytes;
    const char *src = cache + ((long)n * cache_pitch + step) * row_bytes + at;
    char *dst = pool + slot * row_bytes + at;
    const long left = row_bytes - at;
    u32x4 w[kCommitLoads];
    const int size = (int)min(left, (long)kCommitBytes);
    const __amdgpu_buffer_rsrc_t from = __builtin_amdgcn_make_buffer_rsrc(const_cast<char *>(src), 0, size, kBufferWord3);
    const __amdgpu_buffer_rsrc_t to = __builtin_amdgcn_make_buffer_rsrc(dst, 0, size, kBufferWord3);
    const unsigned o = threadIdx.x * 16;
#pragma unroll
    for (int i = 0; i < kCommitLoads; ++i) w[i] = __builtin_amdgcn_raw_buffer_load_b128(from, o + i * 4096, 0, kPassCaches);
#pragma unroll
    for (int i = 0; i < kCommitLoads; ++i) __builtin_amdgcn_raw_buffer_store_b128(w[i], to, o + i * 4096, 0, kPassCaches);
}

hipError_t launch_commit(const int32_t *indices, const int32_t *steps, const void *cache, void *pool, int num_seqs, int num_slots,
                         int cache_steps, int cache_pitch, long row_bytes, hipStream_t s) {
    const dim3 grid((unsigned)((row_bytes + kCommitBytes - 1) / kCommitBytes), decode_grid_y(num_seqs), decode_grid_z(num_seqs));
    commit_kernel<<<grid, 256, 0, s>>>(indices, steps, static_cast<const char *>(cache), static_cast<char *>(pool), num_seqs,
                                       num_slots, cache_steps, cache_pitch, row_bytes);
    return hipGetLastError();
}

}  // namespace kda
