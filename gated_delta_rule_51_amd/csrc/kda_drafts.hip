// Verification of drafted tokens against the target's probabilities, and the
// commit of the accepted states.
//
// A request's drafts are tested 64 at a time, one a lane; the first refused
// one gives the row whose rest the next token is drawn from.  That row (and
// the drafts' own, where one was refused) is read once: wave-sized parts are
// summed in fp64, the part that holds r times the total is found from the
// sums, and only that part is read again to find the token.  Bound by those
// rows' bytes with many requests, by the chain of dependent loads with one.
#include "kda_device.h"
#include "kda_internal.h"

namespace kda {

constexpr int kVerifyWaves = 8;                    // waves (parts) of a workgroup
constexpr int kVerifyThreads = kVerifyWaves * 64;
constexpr int kVerifyParts = 256;                  // most parts of a row

// Parts a row is summed in.  One workgroup's waves where the requests fill the
// chip by themselves; else more workgroups a row, no part below 1024 tokens.
int verify_parts(int num_seqs, int vocab) {
    int parts = kVerifyWaves;
    while (parts < kVerifyParts && (long)num_seqs * parts < 4096 && vocab / (2 * parts) >= 1024) parts *= 2;
    return parts;
}

struct Verdict {
    int t0, len, accepted;   // accepted: drafts that stood
    int wrong;               // the refused draft, or -1 where every one stood
    bool refused;
};

template <typename PT> __device__ __forceinline__ Verdict judge(const VerifyArgs &a, int n, int lane) {
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

// The weight of token i in the refused row (or the last one), and p itself.
template <typename PT> struct Row {
    const PT *p, *q;   // q: NULL where nothing is taken off
    int wrong;         // token of weight 0, or -1
    __device__ __forceinline__ void at(int i, float &w, float &own) const {
        const float x = io_traits<PT>::load(p, i);
        own = fmaxf(x, 0.f);   // NaN weighs nothing
        w = q ? fmaxf(x - io_traits<PT>::load(q, i), 0.f) : i == wrong ? 0.f : own;
    }
};

template <typename PT> __device__ __forceinline__ Row<PT> row_of(const VerifyArgs &a, const Verdict &v) {
    const long t = v.t0 + v.accepted;
    Row<PT> r;
    r.p = reinterpret_cast<const PT *>(a.target) + t * a.target_stride;
    r.q = a.draft && v.refused ? reinterpret_cast<const PT *>(a.draft) + t * a.draft_stride : nullptr;
    r.wrong = v.refused ? v.wrong : -1;
    return r;
}

__device__ __forceinline__ double wave_sum(double x) {
#pragma unroll
    for (int m = 32; m >= 1; m >>= 1) x += __shfl_xor(x, m, 64);
    return x;
}

// Range of part k of `parts`: whole multiples of 64 tokens but for the last.
__device__ __forceinline__ void part_range(int vocab, int parts, int k, int &lo, int &hi) {
    const int each = ((vocab + parts - 1) / parts + 63) / 64 * 64;
    lo = (int)min((long)vocab, (long)each * k);
    hi = (int)min((long)vocab, (long)lo + each);
}

template <typename PT>
__device__ __forceinline__ void sum_part(const Row<PT> &r, int lo, int hi, int lane, double &w, double &own) {
    w = 0.0;
    own = 0.0;
    for (int i = lo + lane; i < hi; i += 64) {
        float x, o;
        r.at(i, x, o);
        w += (double)x;
        own += (double)o;
    }
    w = wave_sum(w);
    own = wave_sum(own);
}

// The whole workgroup: the sums of all parts are in sums[0][..] (weights) and
// sums[1][..] (p); writes the request's outputs.
template <typename PT>
__device__ void pick(const VerifyArgs &a, int n, const Verdict &v, const Row<PT> &r, const double *sums, double *scan) {
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int parts = a.parts;
    __shared__ int found;
    // every thread walks the sums alike: no part to agree on
    double total = 0.0;
    for (int k = 0; k < parts; ++k) total += sums[k];
    const bool rest = total > 0.0;
    if (!rest) {
        total = 0.0;
        for (int k = 0; k < parts; ++k) total += sums[parts + k];
    }
    const double *s = rest ? sums : sums + parts;
    const double want = (double)a.uniform_next[n] * total;
    double before = 0.0, cum = 0.0;
    int part = -1;
    for (int k = 0; k < parts; ++k) {
        if (s[k] > 0.0) {   // the last part with any weight where none reaches past `want`
            part = k;
            before = cum;
        }
        cum += s[k];
        if (cum > want) break;
    }
    if (tid == 0) found = -1;
    __syncthreads();
    if (part >= 0) {
        int lo, hi;
        part_range(a.vocab, parts, part, lo, hi);
        double carry = before;
        for (int base = lo; base < hi; base += kVerifyThreads) {
            const int i = base + tid;
            float w = 0.f, own = 0.f;
            if (i < hi) r.at(i, w, own);
            const double x = rest ? (double)w : (double)own;
            double c = x;
#pragma unroll
            for (int m = 1; m < 64; m <<= 1) {
                const double y = __shfl_up(c, m, 64);
                if (lane >= m) c += y;
            }
            if (lane == 63) scan[wave] = c;
            __syncthreads();
            double off = carry;
            for (int k = 0; k < wave; ++k) off += scan[k];
            for (int k = 0; k < kVerifyWaves; ++k) carry += scan[k];
            // the first token past `want`; failing that (rounding, or a random
            // number of 1) the last token with any weight
            const unsigned long long past = __ballot(x > 0.0 && off + c > want);
            if (past && lane == 0) scan[kVerifyWaves + wave] = (double)(base + wave * 64 + __builtin_ctzll(past));
            else if (lane == 0) scan[kVerifyWaves + wave] = -1.0;
            const unsigned long long some = __ballot(x > 0.0);
            if (lane == 0) scan[2 * kVerifyWaves + wave] = some ? (double)(base + wave * 64 + 63 - __builtin_clzll(some)) : -1.0;
            __syncthreads();
            int hit = -1, last = -1;
            for (int k = 0; k < kVerifyWaves; ++k) {
                if (hit < 0 && scan[kVerifyWaves + k] >= 0.0) hit = (int)scan[kVerifyWaves + k];
                if (scan[2 * kVerifyWaves + k] >= 0.0) last = (int)scan[2 * kVerifyWaves + k];
            }
            if (tid == 0 && (hit >= 0 || last >= 0)) found = hit >= 0 ? hit : last;
            __syncthreads();
            if (hit >= 0) break;
        }
    }
    __syncthreads();
    const int next = found;
    if (tid == 0) {
        a.accepted[n] = v.accepted;
        a.next[n] = next;
    }
    for (int j = tid; j < v.len; j += kVerifyThreads)
        a.emitted[v.t0 + j] = j < v.accepted ? a.tokens[v.t0 + j + 1] : j == v.accepted ? next : -1;
}

// grid (workgroups of a row, requests on y and z): sums the parts; with one
// workgroup a row also finds the token.
template <typename PT> __global__ __launch_bounds__(kVerifyThreads) void verify_sum_kernel(VerifyArgs a) {
    __shared__ double sums[2 * kVerifyWaves], scan[3 * kVerifyWaves];
    const int n = (int)blockIdx.y + (int)blockIdx.z * (int)gridDim.y;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    if (n >= a.num_seqs) return;
    const Verdict v = judge<PT>(a, n, lane);
    if (v.len <= 0) {
        if (blockIdx.x == 0 && threadIdx.x == 0) {
            a.accepted[n] = -1;
            a.next[n] = -1;
        }
        return;
    }
    const Row<PT> r = row_of<PT>(a, v);
    const int part = (int)blockIdx.x * kVerifyWaves + wave;
    int lo, hi;
    part_range(a.vocab, a.parts, part, lo, hi);
    double w, own;
    sum_part<PT>(r, lo, hi, lane, w, own);
    if (gridDim.x > 1) {
        if (lane == 0) {
            a.partial[((long)n * 2) * a.parts + part] = w;
            a.partial[((long)n * 2 + 1) * a.parts + part] = own;
        }
        return;
    }
    if (lane == 0) {
        sums[wave] = w;
        sums[kVerifyWaves + wave] = own;
    }
    __syncthreads();
    pick<PT>(a, n, v, r, sums, scan);
}

// grid (1, requests on y and z): the token from the parts' sums.
template <typename PT> __global__ __launch_bounds__(kVerifyThreads) void verify_pick_kernel(VerifyArgs a) {
    __shared__ double sums[2 * kVerifyParts], scan[3 * kVerifyWaves];
    const int n = (int)blockIdx.y + (int)blockIdx.z * (int)gridDim.y;
    if (n >= a.num_seqs) return;
    for (int k = threadIdx.x; k < 2 * a.parts; k += kVerifyThreads) sums[k] = a.partial[(long)n * 2 * a.parts + k];
    const Verdict v = judge<PT>(a, n, threadIdx.x & 63);
    if (v.len <= 0) return;
    __syncthreads();
    pick<PT>(a, n, v, row_of<PT>(a, v), sums, scan);
}

template <typename PT> static hipError_t launch_p(const VerifyArgs &a, hipStream_t s) {
    const dim3 grid(a.parts / kVerifyWaves, decode_grid_y(a.num_seqs), decode_grid_z(a.num_seqs));
    verify_sum_kernel<PT><<<grid, kVerifyThreads, 0, s>>>(a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || grid.x == 1) return e;
    verify_pick_kernel<PT><<<dim3(1, grid.y, grid.z), kVerifyThreads, 0, s>>>(a);
    return hipGetLastError();
}
hipError_t launch_verify(const VerifyArgs &a, hipStream_t s) { return a.bf16 ? launch_p<bf16>(a, s) : launch_p<float>(a, s); }

// ---- commit ----------------------------------------------------------------

constexpr int kCommitBytes = 256 * 16 * 8;   // bytes of a workgroup: eight 16-byte accesses a thread

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
    const long at = (long)blockIdx.x * kCommitBytes + (long)threadIdx.x * 16;
    const char *src = cache + ((long)n * cache_pitch + step) * row_bytes + at;
    char *dst = pool + slot * row_bytes + at;
    const long left = row_bytes - at;
    u32x4 w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (i * 4096L < left) w[i] = __builtin_nontemporal_load(reinterpret_cast<const u32x4 *>(src + i * 4096L));
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (i * 4096L < left) __builtin_nontemporal_store(w[i], reinterpret_cast<u32x4 *>(dst + i * 4096L));
}

hipError_t launch_commit(const int32_t *indices, const int32_t *steps, const void *cache, void *pool, int num_seqs, int num_slots,
                         int cache_steps, int cache_pitch, long row_bytes, hipStream_t s) {
    const dim3 grid((unsigned)((row_bytes + kCommitBytes - 1) / kCommitBytes), decode_grid_y(num_seqs), decode_grid_z(num_seqs));
    commit_kernel<<<grid, 256, 0, s>>>(indices, steps, static_cast<const char *>(cache), static_cast<char *>(pool), num_seqs,
                                       num_slots, cache_steps, cache_pitch, row_bytes);
    return hipGetLastError();
}

}  // namespace kda
