// Block tables and slot maps from request lengths, on the GPU.
//
// Request n holds len tokens in `held` blocks and is to take L more, so it
// needs max(0, ceil((len + L) / b) - held) blocks.  With P_n the inclusive
// sum of the needs in the batch's order, its j-th new block is entry
// count - 1 - (P_n - need_n + j) of the free list, a stack, as long as
// P_n <= count.  A release pushes the blocks in the opposite order, so giving
// back what the last call took restores the list.
//
// Bound by latency: N + T words are read and written.  One workgroup takes
// the whole batch, since the stack's top is one number for all of it; the
// slots of many tokens follow in a launch of their own over the whole chip.
// 256 requests with a token each 5.2 us, 96 prompts with 129,600 slots 5.0 and
// 4.0, a release 5.2: four dependent reads and two scans.
#include "kda_device.h"
#include "kda_internal.h"

namespace kda {
namespace {

constexpr int kThreads = 1024, kWaves = kThreads / 64;
constexpr uint32_t kMost = 0x7fffffffu;

// Sums that stay at kMost once they pass it (associative, as all terms are at
// most kMost): a batch may ask for more than 2^31 blocks, none of which exist.
__device__ __forceinline__ uint32_t sat_add(uint32_t a, uint32_t b) { return min(a + b, kMost); }

// Exclusive sums over the workgroup's threads; `all` their total.
__device__ __forceinline__ uint32_t block_scan(uint32_t x, uint32_t *parts, uint32_t &all) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    uint32_t incl = x;
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) {
        const uint32_t y = __shfl_up(incl, m, 64);
        if (lane >= m) incl = sat_add(incl, y);
    }
    if (lane == 63) parts[wave] = incl;
    __syncthreads();
    uint32_t before = 0, total = 0;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
        const uint32_t p = parts[w];
        if (w < wave) before = sat_add(before, p);
        total = sat_add(total, p);
    }
    __syncthreads();
    all = total;
    const uint32_t up = __shfl_up(incl, 1, 64);
    return sat_add(before, lane ? up : 0);
}

__device__ __forceinline__ int row_of(const PagesArgs &a, int n) {
    const int r = a.indices[n];
    return (unsigned)r < (unsigned)a.rows ? r : -1;
}

// The last i in [0, n) with at[i] <= x (at[0] <= x).
template <typename T> __device__ __forceinline__ int last_up_to(const T *at, int n, T x) {
    int lo = 0;
    while (n > 1) {
        const int half = n >> 1;
        if (at[lo + half] <= x) {
            lo += half;
            n -= half;
        } else {
            n = half;
        }
    }
    return lo;
}

__device__ __forceinline__ int slot_in(int block, int off, int shift) {
    const long s = ((long)block << shift) + off;
    return block < 0 || s > INT32_MAX ? -1 : (int)s;
}

template <bool SLOTS> __global__ __launch_bounds__(kThreads) void reserve_kernel(const PagesArgs a) {
    __shared__ uint32_t parts[kWaves];
    __shared__ uint32_t first[kThreads];   // new blocks before this request's
    __shared__ int start[kThreads], row[kThreads], held[kThreads], length[kThreads];
    const int tid = threadIdx.x, b = 1 << a.block_shift;
    const uint32_t count = (uint32_t)min(max(a.free_count[0], 0), a.num_free);
    uint32_t asked = 0, taken = 0;
    for (long first_n = 0; first_n < a.num_seqs; first_n += kThreads) {
        const int n0 = (int)first_n;
        const int n = n0 + tid, some = min(kThreads, a.num_seqs - n0);
        int r = -1, have = 0, len = 0, begin = 0;
        long want = 0, total = 0;
        if (n < a.num_seqs) {
            r = row_of(a, n);
            begin = a.cu_seqlens[n];
            const int more = max(a.cu_seqlens[n + 1] - begin, 0);
            if (r >= 0) {
                len = max(a.kv_lens[r], 0);
                have = min(max(a.blocks_held[r], 0), a.max_blocks);
                total = (long)len + more;
                want = (total + b - 1) >> a.block_shift;
                if (want > a.max_blocks || total > INT32_MAX) r = -1;
            }
        }
        const uint32_t need = r >= 0 && want > have ? (uint32_t)(want - have) : 0;
        uint32_t sum;
        const uint32_t before = sat_add(asked, block_scan(need, parts, sum));
        const bool given = r >= 0 && (need == 0 || sat_add(before, need) <= count);
        asked = sat_add(asked, sum);
        // once a request does not fit none behind it takes any, so what is taken so far is a prefix of what is asked for
        uint32_t got;
        block_scan(given ? need : 0, parts, got);
        if (n < a.num_seqs) {
            a.kv_totals[n] = given ? (int)total : 0;
            if (given && need) a.blocks_held[r] = have + (int)need;
        }
        first[tid] = before;
        start[tid] = begin;
        row[tid] = given ? r : -1;
        held[tid] = have;
        length[tid] = len;
        __syncthreads();
        for (uint32_t i = tid; i < got; i += kThreads) {   // the new entries of the tables
            const int k = last_up_to(first, some, taken + i);
            a.block_table[(long)row[k] * a.max_blocks + held[k] + (int)(taken + i - first[k])] = a.free_blocks[count - 1 - (taken + i)];
        }
        if constexpr (SLOTS) {
            const int t0 = max(start[0], 0), t1 = min(a.cu_seqlens[n0 + some], a.total_tokens);
            for (int t = t0 + tid; t < t1; t += kThreads) {
                const int k = last_up_to(start, some, t), pos = length[k] + t - start[k], j = pos >> a.block_shift;
                int block = -1;
                if (row[k] >= 0) {
                    const uint32_t at = first[k] + (uint32_t)(j - held[k]);
                    if (j < held[k]) block = a.block_table[(long)row[k] * a.max_blocks + j];
                    else if (at < count) block = a.free_blocks[count - 1 - at];
                }
                a.slots[t] = slot_in(block, pos & (b - 1), a.block_shift);
            }
        }
        taken += got;
        __syncthreads();
    }
    if constexpr (SLOTS) {
        const int end = max(a.num_seqs ? a.cu_seqlens[a.num_seqs] : 0, 0);
        for (int t = end + tid; t < a.total_tokens; t += kThreads) a.slots[t] = -1;
    }
    if (tid == 0) a.free_count[0] = (int)(count - taken);
}

// Slots of many tokens, from the tables that are written by then.
__global__ __launch_bounds__(256) void slots_kernel(const PagesArgs a) {
    const int t = blockIdx.x * 256 + threadIdx.x;
    if (t >= a.total_tokens) return;
    int slot = -1;
    if (a.num_seqs && t >= a.cu_seqlens[0] && t < a.cu_seqlens[a.num_seqs]) {
        const int n = last_up_to(a.cu_seqlens, a.num_seqs, t), end = a.cu_seqlens[n + 1], total = a.kv_totals[n];
        const int pos = total - (end - t), r = row_of(a, n);
        if (r >= 0 && total > 0 && pos >= 0)
            slot = slot_in(a.block_table[(long)r * a.max_blocks + (pos >> a.block_shift)], pos & ((1 << a.block_shift) - 1), a.block_shift);
    }
    a.slots[t] = slot;
}

__global__ __launch_bounds__(kThreads) void release_kernel(const PagesArgs a) {
    __shared__ uint32_t parts[kWaves], first[kThreads];
    __shared__ int row[kThreads], left[kThreads];
    const int tid = threadIdx.x, b = 1 << a.block_shift;
    const uint32_t count = (uint32_t)min(max(a.free_count[0], 0), a.num_free);
    uint32_t all = 0, before = 0, top = 0;
    for (int pass = 0; pass < 2; ++pass) {   // how many there are, then where each goes
        for (long first_n = 0; first_n < a.num_seqs; first_n += kThreads) {
            const int n0 = (int)first_n;
            const int n = n0 + tid, some = min(kThreads, a.num_seqs - n0);
            int r = -1, keep = 0, stay = 0;
            uint32_t give = 0;
            if (n < a.num_seqs && (r = row_of(a, n)) >= 0) {
                keep = max(a.kv_lens[r], 0);
                if (a.keep_lens) keep = min(keep, max(a.keep_lens[n], 0));
                else keep = 0;
                stay = (int)(((long)keep + b - 1) >> a.block_shift);
                give = (uint32_t)max(min(max(a.blocks_held[r], 0), a.max_blocks) - stay, 0);
            }
            uint32_t sum;
            const uint32_t at = sat_add(before, block_scan(give, parts, sum));
            if (pass) {
                if (r >= 0) {
                    a.kv_lens[r] = keep;
                    if (give) a.blocks_held[r] = stay;
                }
                first[tid] = at;
                row[tid] = r;
                left[tid] = stay;
                __syncthreads();
                for (uint32_t i = tid; i < sum; i += kThreads) {
                    const int k = last_up_to(first, some, before + i);
                    const uint32_t to = top - 1 - (before + i);
                    if (to < (uint32_t)a.num_free)
                        a.free_blocks[to] = a.block_table[(long)row[k] * a.max_blocks + left[k] + (int)(before + i - first[k])];
                }
                __syncthreads();
            }
            before = sat_add(before, sum);
        }
        if (!pass) {
            all = before;
            before = 0;
            top = sat_add(count, all);
        }
    }
    if (tid == 0) a.free_count[0] = (int)min(top, (uint32_t)a.num_free);
}

__global__ __launch_bounds__(256) void commit_kernel(const PagesArgs a) {
    const int n = blockIdx.x * 256 + threadIdx.x;
    if (n >= a.num_seqs) return;
    const int r = row_of(a, n), L = a.cu_seqlens[n + 1] - a.cu_seqlens[n];
    if (r < 0) return;
    const int s = a.steps ? a.steps[n] : L - 1;
    if (s < 0 || s >= L) return;
    // a reservation gives blocks to a request's run as a whole or not at all, and only then were its tokens stored
    const long len = max(a.kv_lens[r], 0);   // as the reservation counts it
    if (len + L <= min((long)a.blocks_held[r] << a.block_shift, (long)INT32_MAX)) a.kv_lens[r] = (int)(len + s + 1);
}

}  // namespace

// Up to this many tokens the workgroup that holds the tables writes the slots
// too.
constexpr int kSlotsAtOnce = 8192;

// Workgroups of 256 for n items, up to 2^31 - 1 of them.
static unsigned groups_of(int n) { return (unsigned)(((long)n + 255) / 256); }

hipError_t launch_reserve(const PagesArgs &a, hipStream_t stream) {
    if (a.total_tokens <= kSlotsAtOnce) {
        reserve_kernel<true><<<1, kThreads, 0, stream>>>(a);
        return hipGetLastError();
    }
    reserve_kernel<false><<<1, kThreads, 0, stream>>>(a);
    slots_kernel<<<groups_of(a.total_tokens), 256, 0, stream>>>(a);
    return hipGetLastError();
}

hipError_t launch_release(const PagesArgs &a, hipStream_t stream) {
    release_kernel<<<1, kThreads, 0, stream>>>(a);
    return hipGetLastError();
}

hipError_t launch_kv_commit(const PagesArgs &a, hipStream_t stream) {
    commit_kernel<<<groups_of(a.num_seqs), 256, 0, stream>>>(a);
    return hipGetLastError();
}

}  // namespace kda
