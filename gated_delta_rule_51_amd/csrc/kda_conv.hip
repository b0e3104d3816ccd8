// Short causal depthwise convolution with SiLU, over packed prompts, for one
// token a request, and the commit of accepted inputs to the pool.
//
//     s[t, c] = bias[c] + sum_{j < W} weight[c, j] x[t - W + 1 + j, c],   y = s / (1 + e^-s)
//
// A state is the last W - 1 raw inputs [W - 1, D], oldest first, D contiguous,
// so that every tap is a coalesced row like those of x.  2 W + 4 operations
// an element against 2 elements of traffic: bound by memory.  Each thread
// holds VEC neighbouring channels (16 bytes where rows allow it, else one) and
// slides a window of W - 1 rows in registers, so x is read once.
#include "kda_device.h"
#include "kda_internal.h"

namespace kda {

// Tokens per workgroup row of the prefill (the W - 1 rows before it are read
// again, from the caches) and rows loaded ahead.  30,447 tokens x 6144 channels
// (bf16, four taps; 0.75 GB), y stored past the caches: 16 tokens by 8 rows
// 132 us (5.7 TB/s), by 16 134, 8 by 8 135, 32 by 16 136; with ordinary stores
// 16 by 16 147, 32 by 4 160, 64 by 4 174.  Rows that are no multiple of 16 bytes
// go one channel a thread: 6143 channels 177 us (4.2 TB/s); in fp32 320 us against
// 265 for 6144.
constexpr int kConvTile = 16, kConvAhead = 8;

long conv_prefill_tiles(int num_seqs, int total_tokens) {
    return num_seqs <= 0 ? 0 : (long)total_tokens / kConvTile + num_seqs;
}

// Load / store VEC consecutive elements (16 bytes, or one element).
template <typename IO, int VEC> __device__ __forceinline__ void load_v(const IO *p, float (&r)[VEC]) {
    if constexpr (VEC == 1) {
        r[0] = io_traits<IO>::load(p, 0);
    } else {
#pragma unroll
        for (int i = 0; i < VEC; i += 4) {
            const f32x4 x = load4(p + i);
#pragma unroll
            for (int e = 0; e < 4; ++e) r[i + e] = x[e];
        }
    }
}
template <typename IO, int VEC, bool NT = false> __device__ __forceinline__ void store_v(IO *p, const float (&r)[VEC]) {
    if constexpr (VEC == 1) {
        io_traits<IO>::store(p, 0, r[0]);
    } else if constexpr (VEC == 4) {
        const f32x4 w = {r[0], r[1], r[2], r[3]};
        if constexpr (NT) __builtin_nontemporal_store(w, reinterpret_cast<f32x4 *>(p));
        else *reinterpret_cast<f32x4 *>(p) = w;
    } else {
        u32x4 w;
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = pack_bf16x2(r[2 * i], r[2 * i + 1]);
        if constexpr (NT) __builtin_nontemporal_store(w, reinterpret_cast<u32x4 *>(p));
        else *reinterpret_cast<u32x4 *>(p) = w;
    }
}

// The taps and bias of this thread's channels: wt[j][e] = weight[c + e, j].
template <typename IO, int VEC, int W>
__device__ __forceinline__ void load_taps(const ConvArgs &a, int c, float (&wt)[W][VEC], float (&bs)[VEC]) {
    const IO *wp = reinterpret_cast<const IO *>(a.weight) + (long)c * W;
#pragma unroll
    for (int e = 0; e < VEC; ++e)
#pragma unroll
        for (int j = 0; j < W; ++j) wt[j][e] = io_traits<IO>::load(wp, e * W + j);
#pragma unroll
    for (int e = 0; e < VEC; ++e) bs[e] = a.bias ? io_traits<IO>::load(reinterpret_cast<const IO *>(a.bias), c + e) : 0.f;
}

// s / (1 + e^-s); e^-s overflowing gives -0.
__device__ __forceinline__ float silu_f(float s) { return s * sigmoid_f(s); }

template <int VEC, int W>
__device__ __forceinline__ void conv_out(const float (&win)[W - 1][VEC], const float (&cur)[VEC], const float (&wt)[W][VEC],
                                         const float (&bs)[VEC], bool silu, float (&y)[VEC]) {
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
        float s = bs[e];
#pragma unroll
        for (int j = 0; j < W - 1; ++j) s += wt[j][e] * win[j][e];
        s += wt[W - 1][e] * cur[e];
        y[e] = silu ? silu_f(s) : s;
    }
}

// grid (channel blocks, tile slots on y and z)
template <typename IO, int VEC, int W> __global__ __launch_bounds__(256) void conv_prefill_kernel(ConvArgs a, int slots) {
    const int slot = (int)blockIdx.y + (int)blockIdx.z * (int)gridDim.y;
    const int c = ((int)blockIdx.x * 256 + (int)threadIdx.x) * VEC;
    if (slot >= slots) return;
    const int n = slot_sequence(a.cu_seqlens, a.num_seqs, slot, kConvTile);
    const int begin = a.cu_seqlens[n], len = a.cu_seqlens[n + 1] - begin;
    const int local = (slot - (begin / kConvTile + n)) * kConvTile;   // first token of the tile
    if (c >= a.channels || (local >= len && local > 0)) return;

    const long D = a.channels;
    const IO *x = reinterpret_cast<const IO *>(a.x) + (long)begin * a.x_stride + c;
    float win[W - 1][VEC];
    if (local == 0) {
        long row = n;
        if (a.indices) {
            row = a.indices[n];
            if (row < 0) row = a.num_slots - 1;
        }
        const long at = row * (W - 1) * D + c;
#pragma unroll
        for (int j = 0; j < W - 1; ++j) {
            if (a.state_in) {
                load_v<IO, VEC>(reinterpret_cast<const IO *>(a.state_in) + at + j * D, win[j]);
            } else {
#pragma unroll
                for (int e = 0; e < VEC; ++e) win[j][e] = 0.f;
            }
        }
        // The last inputs are written here, by the only thread that reads the
        // state (in place in a pool): row j is input len + j of (state, x).
        if (a.state_out && !(a.indices && len <= 0)) {
#pragma unroll
            for (int j = 0; j < W - 1; ++j) {
                float r[VEC];
                const int k = len + j;
                if (k >= W - 1) {
                    load_v<IO, VEC>(x + (long)(k - (W - 1)) * a.x_stride, r);
                } else {
#pragma unroll
                    for (int e = 0; e < VEC; ++e) {
                        r[e] = win[0][e];
#pragma unroll
                        for (int i = 1; i < W - 1; ++i) r[e] = k == i ? win[i][e] : r[e];
                    }
                }
                store_v<IO, VEC>(reinterpret_cast<IO *>(a.state_out) + at + j * D, r);
            }
        }
        if (len <= 0) return;
    } else {
#pragma unroll
        for (int j = 0; j < W - 1; ++j) load_v<IO, VEC>(x + (long)(local - (W - 1) + j) * a.x_stride, win[j]);
    }
    float wt[W][VEC], bs[VEC];
    load_taps<IO, VEC, W>(a, c, wt, bs);
    IO *y = reinterpret_cast<IO *>(a.y) + (long)begin * D + c;
    const int end = min(local + kConvTile, len);
    constexpr int U = kConvAhead;
    int t = local;
    for (; t + U <= end; t += U) {
        float cur[U][VEC];
#pragma unroll
        for (int u = 0; u < U; ++u) load_v<IO, VEC>(x + (long)(t + u) * a.x_stride, cur[u]);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float o[VEC];
            conv_out<VEC, W>(win, cur[u], wt, bs, a.silu, o);
            store_v<IO, VEC, true>(y + (long)(t + u) * D, o);
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
#pragma unroll
                for (int j = 0; j + 1 < W - 1; ++j) win[j][e] = win[j + 1][e];
                win[W - 2][e] = cur[u][e];
            }
        }
    }
    for (; t < end; ++t) {
        float cur[VEC], o[VEC];
        load_v<IO, VEC>(x + (long)t * a.x_stride, cur);
        conv_out<VEC, W>(win, cur, wt, bs, a.silu, o);
        store_v<IO, VEC, true>(y + (long)t * D, o);
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
#pragma unroll
            for (int j = 0; j + 1 < W - 1; ++j) win[j][e] = win[j + 1][e];
            win[W - 2][e] = cur[e];
        }
    }
}

// A token of every request: a launch and one load's latency with few (200
// requests x 2051 channels, fp32, three taps: 4.0 us for 10 MB), memory with many
// (4096 x 6144, bf16, four taps: 91 us, 4.5 TB/s; 6143 channels 117).
// grid (channel blocks, requests on y and z)
template <typename IO, int VEC, int W> __global__ __launch_bounds__(256) void conv_decode_kernel(ConvArgs a) {
    const int b = (int)blockIdx.y + (int)blockIdx.z * (int)gridDim.y;
    const int c = ((int)blockIdx.x * 256 + (int)threadIdx.x) * VEC;
    if (b >= a.num_seqs || c >= a.channels) return;
    const long D = a.channels;
    long row = a.indices[b];
    if (row < 0) row = a.num_slots - 1;
    IO *st = reinterpret_cast<IO *>(a.state_out) + row * (W - 1) * D + c;
    float win[W - 1][VEC], cur[VEC], o[VEC], wt[W][VEC], bs[VEC];
#pragma unroll
    for (int j = 0; j < W - 1; ++j) load_v<IO, VEC>(st + j * D, win[j]);
    load_v<IO, VEC>(reinterpret_cast<const IO *>(a.x) + (long)b * a.x_stride + c, cur);
    load_taps<IO, VEC, W>(a, c, wt, bs);
    conv_out<VEC, W>(win, cur, wt, bs, a.silu, o);
    store_v<IO, VEC>(reinterpret_cast<IO *>(a.y) + (long)b * D + c, o);
#pragma unroll
    for (int j = 0; j + 1 < W - 1; ++j) store_v<IO, VEC>(st + j * D, win[j + 1]);
    store_v<IO, VEC>(st + (W - 2) * D, cur);
}

// Row j of the new state is input steps[n] + 1 + j of (state, x): copies.
// 1024 requests x 4096 channels (bf16, four taps) 8.7 us, 5.8 TB/s; three requests 2.8 us.
template <typename IO, int VEC, int W> __global__ __launch_bounds__(256) void conv_commit_kernel(ConvArgs a) {
    const int n = (int)blockIdx.y + (int)blockIdx.z * (int)gridDim.y;
    const int c = ((int)blockIdx.x * 256 + (int)threadIdx.x) * VEC;
    if (n >= a.num_seqs || c >= a.channels) return;
    const int begin = a.cu_seqlens[n], len = a.steps[n] + 1;
    if (len <= 0 || len > a.cu_seqlens[n + 1] - begin) return;
    const long D = a.channels;
    long row = a.indices[n];
    if (row < 0) row = a.num_slots - 1;
    IO *st = reinterpret_cast<IO *>(a.state_out) + row * (W - 1) * D + c;
    const IO *x = reinterpret_cast<const IO *>(a.x) + (long)begin * a.x_stride + c;
    // row j takes a row at or after j: in place, front to back
    float r[W - 1][VEC];
#pragma unroll
    for (int j = 0; j < W - 1; ++j) {
        const int k = len + j;
        if (k >= W - 1) load_v<IO, VEC>(x + (long)(k - (W - 1)) * a.x_stride, r[j]);
        else load_v<IO, VEC>(st + k * D, r[j]);
    }
#pragma unroll
    for (int j = 0; j < W - 1; ++j) store_v<IO, VEC>(st + j * D, r[j]);
}

enum class ConvOp { prefill, decode, commit };

template <typename IO, int VEC, int W> static hipError_t launch_w(const ConvArgs &a, ConvOp op, hipStream_t s) {
    const long rows = op == ConvOp::prefill ? conv_prefill_tiles(a.num_seqs, a.total_tokens) : a.num_seqs;
    const dim3 grid((unsigned)((a.channels + 256L * VEC - 1) / (256L * VEC)), decode_grid_y((int)rows), decode_grid_z((int)rows));
    switch (op) {
    case ConvOp::prefill: conv_prefill_kernel<IO, VEC, W><<<grid, 256, 0, s>>>(a, (int)rows); break;
    case ConvOp::decode: conv_decode_kernel<IO, VEC, W><<<grid, 256, 0, s>>>(a); break;
    case ConvOp::commit: conv_commit_kernel<IO, VEC, W><<<grid, 256, 0, s>>>(a); break;
    }
    return hipGetLastError();
}
template <typename IO, int VEC> static hipError_t launch_v(const ConvArgs &a, ConvOp op, hipStream_t s) {
    switch (a.width) {
    case 2: return launch_w<IO, VEC, 2>(a, op, s);
    case 3: return launch_w<IO, VEC, 3>(a, op, s);
    default: return launch_w<IO, VEC, 4>(a, op, s);
    }
}
static hipError_t launch_conv(const ConvArgs &a, ConvOp op, hipStream_t s) {
    // 16-byte accesses need every row 16-byte aligned
    const int vec = a.io_bf16 ? 8 : 4;
    const bool wide = a.channels % vec == 0 && a.x_stride % vec == 0;
    if (a.io_bf16) return wide ? launch_v<bf16, 8>(a, op, s) : launch_v<bf16, 1>(a, op, s);
    return wide ? launch_v<float, 4>(a, op, s) : launch_v<float, 1>(a, op, s);
}

hipError_t launch_conv_prefill(const ConvArgs &a, hipStream_t s) { return launch_conv(a, ConvOp::prefill, s); }
hipError_t launch_conv_decode(const ConvArgs &a, hipStream_t s) { return launch_conv(a, ConvOp::decode, s); }
hipError_t launch_conv_commit(const ConvArgs &a, hipStream_t s) { return launch_conv(a, ConvOp::commit, s); }

}  // namespace kda
