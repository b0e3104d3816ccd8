// What the state-space scan's two prompt kernels (bf16 and fp32 io) share: the
// segments, a workgroup's place among them, a chunk's gates and M.
#pragma once

#include "kda_device.h"
#include "kda_internal.h"
#include "kda_ssm.h"

namespace kda {

typedef float f32x16 __attribute__((ext_vector_type(16)));

// A value (of 8 bytes) all lanes share, in scalar registers.
template <typename T> __device__ __forceinline__ T uniform(T x) {
    static_assert(sizeof(T) == 8, "two registers");
    const u32x2 w = __builtin_bit_cast(u32x2, x);
    return __builtin_bit_cast(T, u32x2{(uint32_t)__builtin_amdgcn_readfirstlane((int)w[0]),
                                       (uint32_t)__builtin_amdgcn_readfirstlane((int)w[1])});
}

struct Segments {
    int len;        // tokens: a multiple of 64, or all of them where every sequence is one segment
    int after;      // floor(T / len): at least the segments after the sequences' first
    bool later;     // the last launch
    // Segment k of sequence n, but for its last, has the place floor(cu[n] / len) + k.
    float *states;  // [after, H, P, S]: after the segment; before the next one once carried
    float *decays;  // [after, H]
};

// The segment and heads of a workgroup of HW heads (of one group).
struct Place {
    int place, seq, t0, len;   // the segment's place, sequence, first token, tokens
    int local, segs;        // number of the segment, segments of the sequence
    int g, first, last;     // group, first head, one past the group's last head
    long row;               // state row (pool slot or sequence)
    bool skip;              // nothing to do in this launch
    bool whole;             // forms y, not the state alone

    __device__ __forceinline__ Place(const SsmArgs &a, const Segments &sg, int hw) {
        const int rep = a.heads / a.groups, blocks = (rep + hw - 1) / hw;
        const int unit = (int)blockIdx.x / (a.groups * blocks), rest = (int)blockIdx.x % (a.groups * blocks);
        g = rest / blocks;
        first = g * rep + rest % blocks * hw;
        last = (g + 1) * rep;
        // The first launch starts with every sequence's first segment, the
        // longer work; the other units are the segments after the first.
        const bool head = !sg.later && unit < a.num_seqs;
        const int after = sg.later ? unit : unit - a.num_seqs;
        seq = __builtin_amdgcn_readfirstlane(head ? unit : slot_sequence<0>(a.cu_seqlens, a.num_seqs, after, sg.len));
        const int begin = __builtin_amdgcn_readfirstlane(a.cu_seqlens[seq]);
        const int all = __builtin_amdgcn_readfirstlane(a.cu_seqlens[seq + 1]) - begin;
        local = head ? 0 : after - begin / sg.len + 1;
        place = begin / sg.len + local;
        segs = all > 0 ? (all - 1) / sg.len + 1 : 1;
        t0 = begin + local * sg.len;
        len = min(sg.len, all - local * sg.len);
        row = seq;
        whole = sg.later || head;
        skip = !head && (local >= segs || (!sg.later && local == segs - 1));
        skip = skip || (len <= 0 && (a.indices || !a.state_out));
        if (!skip && a.indices) {
            row = a.indices[seq];
            if (row < 0) row = a.num_slots - 1;
        }
    }
};

// Per token of a chunk: 0 and 1 the two floats of G (in powers of 2), 2 dt
// over the decay of the second, 3 exp(G_last - G) dt, 4 exp(G).
constexpr int kGateArrays = 5;

// The gates of a chunk, a token a lane: G is the inclusive sum of step x A (A
// in powers of 2), in fp64.  A token's decay below 2^-1024 counts as that: it
// is zero either way, and G stays small enough for two floats, whatever the
// step.  q points at the lane's place in the arrays.  Returns the sum over the
// chunk.
__device__ __forceinline__ double write_gates(float *q, float step, double A) {
    const double G = wave_scan(fmax((double)step * A, -1024.0)), last = lane_value(G, 63);
    const float gh = (float)G, gl = (float)(G - (double)gh);
    q[0] = gh;
    q[64] = gl;
    q[128] = step * __builtin_amdgcn_exp2f(-gl);
    q[192] = step * __builtin_amdgcn_exp2f((float)(last - G));
    q[256] = __builtin_amdgcn_exp2f(gh);
    return last;
}

// Four columns of M's tile (rows t of 32 tt, columns s of 32 ss) from the
// products C_t . B_s: registers 4q .. 4q + 3.  Every pair has its own
// exponential, as a factor to a common point would overflow.
__device__ __forceinline__ void m_part(const f32x16 &cb, const float *gate, int tt, int ss, int q, int lane, float Dh, float gt,
                                       float lt, float (&v)[4]) {
    const int t = 32 * tt + (lane & 31), s0 = 32 * ss + 8 * q + 4 * (lane >> 5);
    const f32x4 gs = *reinterpret_cast<const f32x4 *>(gate + s0), ds = *reinterpret_cast<const f32x4 *>(gate + 128 + s0);
#pragma unroll
    for (int b = 0; b < 4; ++b) {
        const float x = fmaf(cb[4 * q + b], __builtin_amdgcn_exp2f((gt - gs[b]) + lt) * ds[b], s0 + b == t ? Dh : 0.f);
        v[b] = s0 + b <= t ? x : 0.f;
    }
}

int ssm_head_workgroups(const SsmArgs &a);   // workgroups of a segment
// Units of a launch: the sequences' first segments, and those after them.
inline int ssm_units(const SsmArgs &a, const Segments &sg) { return (sg.later ? 0 : a.num_seqs) + sg.after; }
hipError_t launch_ssm_chunk_f32(const SsmArgs &a, const Segments &sg, hipStream_t s);

}  // namespace kda
