// Selective state-space scan of packed prompts, fp32 io, in chunks of 64 tokens
// on the fp32 matrix cores (a sixteenth of bf16's rate; nothing is rounded):
// the chunk's formulas, the segments and the gates are those of bf16 io.
//
// A 32 x 32 x 2 product takes from a lane one value of row (or column)
// lane & 31 at k = lane / 32 and leaves rows 8a + 4 (lane / 32) + b in its
// registers 4a + b.  So register r of one product's result is an operand of
// the next as it stands, with the k slots {8a + b, 8a + 4 + b}: the state
// (columns n) against C, and M (columns s) against x, 16 products a tile.
// B and x enter the state's product row by row, unchanged.
//
// Bound by the matrix cores: 368 products of 64 cycles a wave and chunk at
// P = S = 128, a wave a SIMD (16 prompts of 512 to 4096 tokens x 32 heads 1.48 ms);
// with few short prompts by the length of a chain: 7 of up to 300 tokens x 8 heads
// x (64 x 64) take 40 us in three launches, two of 19 (a chunk each) and the
// carry's 4.7.
#include "kda_ssm_chunk.h"

namespace kda {

__device__ __forceinline__ f32x16 mfma32(float a, float b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x2f32(a, b, c, 0, 0, 0);
}

template <int P, int S> struct ChunkF {
    static constexpr int WPH = P / 32, HW = 4 / WPH, NT = S / 32;
    static constexpr int PPR = S / 4;          // 16-byte pieces of a row of B
    static constexpr int PB = PPR / 4;         // pieces of B a thread stages
    static constexpr int MBYTES = WPH == 1 ? 0 : 3 * 4096;
    static constexpr int OFF_B = 64 * 512, OFF_C = OFF_B + 64 * 4 * S, OFF_M = OFF_C + 64 * 4 * S;
    static constexpr int OFF_G = OFF_M + HW * MBYTES;
    static constexpr int GBYTES = HW * kGateArrays * 256;
    static constexpr int LDS = OFF_G + 2 * GBYTES;
};

// Byte offset of a row's 16-byte piece: pieces are exchanged within rows, so
// that 16 rows of one piece lie in different banks, and so do 32 columns of
// rows r and r + 4 (the two k of a product).
template <int PPR> __device__ __forceinline__ int piece_at(int row, int piece) {
    const int f = PPR >= 16 ? (row & 3) | ((row & 4) << 1) | ((row & 8) >> 1) : (row >> 1) & 7;
    return row * PPR * 16 + ((piece ^ f) << 4);
}

// A workgroup's segment; without Y its state alone.
template <int P, int S, typename ST, bool Y>
__device__ __forceinline__ void run_segment_f32(const SsmArgs &a, const Segments &sg, const Place &at, unsigned char *lds) {
    using C = ChunkF<P, S>;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int hh = lane >> 5, l32 = lane & 31;
    const int hs = wave / C::WPH, pc = wave % C::WPH;   // head of the workgroup, 32-column block of the head
    const int first = at.first, h = first + hs, t0 = at.t0, len = at.len;
    const bool active = h < at.last;

    // state: register 4a + b of tile nt is column n = 32 nt + 8a + 4 hh + b of row l32
    const long one = (long)a.heads * P * S;
    const long in_head = (long)((active ? h : first) * P + 32 * pc + l32) * S + 4 * hh;
    f32x16 st[C::NT];
#pragma unroll
    for (int nt = 0; nt < C::NT; ++nt)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            f32x4 x = {0.f, 0.f, 0.f, 0.f};
            const long o = in_head + 32 * nt + 8 * q;
            if (sg.later) x = load4(sg.states + (at.place - 1) * one + o);
            else if (a.state_in && at.local == 0) x = load4(reinterpret_cast<const ST *>(a.state_in) + at.row * one + o);
#pragma unroll
            for (int b = 0; b < 4; ++b) st[nt][4 * q + b] = x[b];
        }

    const float *xg = reinterpret_cast<const float *>(a.x) + (long)t0 * a.x_stride + (long)first * P;
    const float *bg = reinterpret_cast<const float *>(a.B) + (long)t0 * a.b_stride + (long)at.g * S;
    const float *cg = reinterpret_cast<const float *>(a.C) + (long)t0 * a.c_stride + (long)at.g * S;
    const float *yg = uniform(reinterpret_cast<const float *>(a.y) + (long)t0 * a.heads * P + (long)h * P + 32 * pc);
    const float *zg = uniform(reinterpret_cast<const float *>(a.z) + (long)t0 * a.z_stride + (long)(active ? h : first) * P + 32 * pc);
    // `each` rows from row `from`; rows past the sequence read as zero and are not written
    auto rows_at = [&](const float *base, long stride, int from, int each) {
        const int rows = __builtin_amdgcn_readfirstlane(max(0, min(each, len - from)));
        return __builtin_amdgcn_make_buffer_rsrc(const_cast<float *>(base + from * stride), 0, (int)(rows * stride * 4), kBufferWord3);
    };
    constexpr int XPASS = 8, BPASS = 256 / C::PPR;   // rows a pass of the workgroup loads
    u32x4 xr[8], br[C::PB], cr[C::PB];
    auto stage = [&](int c0) {
        const unsigned xo = (unsigned)((tid / 32) * (int)a.x_stride + (tid % 32) * 4) * 4;
        const unsigned bo = (unsigned)((tid / C::PPR) * (int)a.b_stride + (tid % C::PPR) * 4) * 4;
        const unsigned co = (unsigned)((tid / C::PPR) * (int)a.c_stride + (tid % C::PPR) * 4) * 4;
        const bool in = first + (tid % 32) * 4 / P < at.last;   // the piece's head is there
#pragma unroll
        for (int i = 0; i < 8; ++i)
            xr[i] = __builtin_amdgcn_raw_buffer_load_b128(rows_at(xg, a.x_stride, c0 + XPASS * i, XPASS), in ? xo : 0x80000000u, 0, 0);
#pragma unroll
        for (int i = 0; i < C::PB; ++i) {
            br[i] = __builtin_amdgcn_raw_buffer_load_b128(rows_at(bg, a.b_stride, c0 + BPASS * i, BPASS), bo, 0, 0);
            if constexpr (Y) cr[i] = __builtin_amdgcn_raw_buffer_load_b128(rows_at(cg, a.c_stride, c0 + BPASS * i, BPASS), co, 0, 0);
        }
    };
    // x: columns of 32-column block w of row r, the blocks exchanged in pairs by rows of 4
    auto x_at = [&](int row, int block) { return row * 512 + ((block ^ ((row >> 2) & 1)) << 7); };
    auto unstage = [&]() {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            *reinterpret_cast<u32x4 *>(lds + x_at(tid / 32 + XPASS * i, tid % 32 / 8) + tid % 8 * 16) = xr[i];
#pragma unroll
        for (int i = 0; i < C::PB; ++i) {
            const int o = piece_at<C::PPR>(tid / C::PPR + BPASS * i, tid % C::PPR);
            *reinterpret_cast<u32x4 *>(lds + C::OFF_B + o) = br[i];
            if constexpr (Y) *reinterpret_cast<u32x4 *>(lds + C::OFF_C + o) = cr[i];
        }
    };

    // gates, by the last wave of each head, a token a lane; an empty sequence has
    // none, and without any token A_log may be NULL
    const bool gates = active && len > 0 && pc == C::WPH - 1;
    const double A = uniform(gates ? -exp((double)a.A_log[h]) * 1.4426950408889634 : 0.0);
    const float bias = gates && a.dt_bias ? a.dt_bias[h] : 0.f, Dh = active && a.D ? a.D[h] : 0.f;
    const float *dg = reinterpret_cast<const float *>(a.dt) + (long)t0 * a.dt_stride + h;
    float dtv = 0.f;
    double through = 0.0;   // log2 of the segment's decay
    auto fetch_dt = [&](int c0) { dtv = dg[(long)min(c0 + lane, len - 1) * a.dt_stride]; };
    auto make_gates = [&](int c0, int buf) {
        float *q = reinterpret_cast<float *>(lds + C::OFF_G + buf * C::GBYTES) + hs * kGateArrays * 64 + lane;
        through = uniform(through + write_gates(q, c0 + lane < len ? softplus_f(dtv + bias) : 0.f, A));
    };
    if (len > 0) {
        if (gates) {
            fetch_dt(0);
            make_gates(0, 0);
            fetch_dt(64);
        }
        stage(0);
    }
    float *const mbase = reinterpret_cast<float *>(lds + C::OFF_M + hs * C::MBYTES) + lane * 4;

    int buf = 0;
    for (int c0 = 0; c0 < len; c0 += 64, buf ^= 1) {
        unstage();
        __syncthreads();
        const float *gate = reinterpret_cast<const float *>(lds + C::OFF_G + buf * C::GBYTES) + hs * kGateArrays * 64;
        stage(c0 + 64);   // past the end there are no rows

        // M's tiles (t, s) = (0, 0), (1, 0), (1, 1): C_t . B_s, then the decays
        auto form_m = [&](int tt, int ss) {
            f32x16 cb;
#pragma unroll
            for (int i = 0; i < 16; ++i) cb[i] = 0.f;
#pragma unroll
            for (int q = 0; q < S / 8; ++q) {
                const f32x4 bo = *reinterpret_cast<const f32x4 *>(lds + C::OFF_B + piece_at<C::PPR>(32 * ss + l32, 2 * q + hh));
                const f32x4 co = *reinterpret_cast<const f32x4 *>(lds + C::OFF_C + piece_at<C::PPR>(32 * tt + l32, 2 * q + hh));
#pragma unroll
                for (int b = 0; b < 4; ++b) cb = mfma32(bo[b], co[b], cb);
            }
            const float gt = gate[32 * tt + l32], lt = gate[64 + 32 * tt + l32];
            f32x16 m;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                float v[4];
                m_part(cb, gate, tt, ss, q, lane, Dh, gt, lt, v);
#pragma unroll
                for (int b = 0; b < 4; ++b) m[4 * q + b] = v[b];
            }
            return m;
        };
        if constexpr (Y && C::WPH > 1) {
            if (active) {
#pragma unroll
                for (int tile = 0; tile < 3; ++tile) {
                    if ((C::WPH == 4 ? tile : tile >> 1) != pc) continue;
                    const f32x16 m = form_m(tile > 0, tile > 1);
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        *reinterpret_cast<f32x4 *>(mbase + tile * 1024 + q * 256) = f32x4{m[4 * q], m[4 * q + 1], m[4 * q + 2], m[4 * q + 3]};
                }
            }
        }
        if (gates && c0 + 64 < len) {
            make_gates(c0 + 64, buf ^ 1);
            fetch_dt(c0 + 128);
        }

        // y = exp(G) S C
        f32x16 y[2];
#pragma unroll
        for (int i = 0; i < 16; ++i) y[0][i] = y[1][i] = 0.f;
        if constexpr (Y) {
#pragma unroll
            for (int nt = 0; nt < C::NT; ++nt)
#pragma unroll
                for (int q = 0; q < 4; ++q)
#pragma unroll
                    for (int tt = 0; tt < 2; ++tt) {
                        const f32x4 co = *reinterpret_cast<const f32x4 *>(lds + C::OFF_C + piece_at<C::PPR>(32 * tt + l32, 8 * nt + 2 * q + hh));
#pragma unroll
                        for (int b = 0; b < 4; ++b) y[tt] = mfma32(st[nt][4 * q + b], co[b], y[tt]);
                    }
#pragma unroll
            for (int tt = 0; tt < 2; ++tt) {
                const float e = gate[256 + 32 * tt + l32];
#pragma unroll
                for (int i = 0; i < 16; ++i) y[tt][i] *= e;
            }
        }
        const float all = gate[256 + 63];
#pragma unroll
        for (int nt = 0; nt < C::NT; ++nt)
#pragma unroll
            for (int i = 0; i < 16; ++i) st[nt][i] *= all;
        if constexpr (Y && C::WPH > 1) __syncthreads();   // M is there

        // y += M x: register 4q + b of M against tokens 8q + 4 hh + b
        if constexpr (Y) {
#pragma unroll
            for (int tile = 0; tile < 3; ++tile) {
                const int tt = tile > 0, ss = tile > 1;
                f32x16 m;
                if constexpr (C::WPH == 1) {
                    m = form_m(tt, ss);
                } else {
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const f32x4 v = *reinterpret_cast<const f32x4 *>(mbase + tile * 1024 + q * 256);
#pragma unroll
                        for (int b = 0; b < 4; ++b) m[4 * q + b] = v[b];
                    }
                }
#pragma unroll
                for (int q = 0; q < 4; ++q)
#pragma unroll
                    for (int b = 0; b < 4; ++b) {
                        const float x = *reinterpret_cast<const float *>(lds + x_at(32 * ss + 8 * q + 4 * hh + b, wave) + 4 * l32);
                        y[tt] = mfma32(x, m[4 * q + b], y[tt]);
                    }
            }
        }
        // S += (weights x) B^T, tokens 8q + b and 8q + 4 + b at a time
#pragma unroll 2
        for (int q = 0; q < 8; ++q) {
            const f32x4 w = *reinterpret_cast<const f32x4 *>(gate + 192 + 8 * q + 4 * hh);
#pragma unroll
            for (int b = 0; b < 4; ++b) {
                const int row = 8 * q + 4 * hh + b;
                const float x = *reinterpret_cast<const float *>(lds + x_at(row, wave) + 4 * l32) * w[b];
#pragma unroll
                for (int nt = 0; nt < C::NT; ++nt) {
                    const float bo = *reinterpret_cast<const float *>(lds + C::OFF_B + piece_at<C::PPR>(row, 8 * nt + l32 / 4) + l32 % 4 * 4);
                    st[nt] = mfma32(bo, x, st[nt]);
                }
            }
        }

        if (Y && active) {
#pragma unroll
            for (int tt = 0; tt < 2; ++tt) {
                const __amdgpu_buffer_rsrc_t ys = rows_at(yg, (long)a.heads * P, c0 + 32 * tt, 32);
                const unsigned yo = (unsigned)(l32 * a.heads * P + 4 * hh) * 4, zo = (unsigned)(l32 * (int)a.z_stride + 4 * hh) * 4;
                if (a.z) {
                    const __amdgpu_buffer_rsrc_t zs = rows_at(zg, a.z_stride, c0 + 32 * tt, 32);
                    u32x4 z[4];
#pragma unroll
                    for (int q = 0; q < 4; ++q) z[q] = __builtin_amdgcn_raw_buffer_load_b128(zs, zo + 32 * q, 0, 0);
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const float v = __uint_as_float(z[i / 4][i % 4]);
                        y[tt][i] *= v * sigmoid_f(v);
                    }
                }
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    u32x4 w;
#pragma unroll
                    for (int b = 0; b < 4; ++b) w[b] = __float_as_uint(y[tt][4 * q + b]);
                    __builtin_amdgcn_raw_buffer_store_b128(w, ys, yo + 32 * q, 0, 0);
                }
            }
        }
        __syncthreads();   // every wave has read this chunk
    }

    const bool last = at.local == at.segs - 1;   // else the state goes to the segment's place
    if (!active || (last ? !a.state_out : sg.later)) return;
    if (!last && gates && lane == 0) sg.decays[(long)at.place * a.heads + h] = __builtin_amdgcn_exp2f((float)through);
#pragma unroll
    for (int nt = 0; nt < C::NT; ++nt)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            f32x4 x;
#pragma unroll
            for (int b = 0; b < 4; ++b) x[b] = st[nt][4 * q + b];
            const long o = in_head + 32 * nt + 8 * q;
            if (!last) *reinterpret_cast<f32x4 *>(sg.states + at.place * one + o) = x;
            else if constexpr (sizeof(ST) == 4) *reinterpret_cast<f32x4 *>(reinterpret_cast<ST *>(a.state_out) + at.row * one + o) = x;
            else *reinterpret_cast<u32x2 *>(reinterpret_cast<ST *>(a.state_out) + at.row * one + o) = u32x2{pack2(x[0], x[1]), pack2(x[2], x[3])};
        }
}

template <int P, int S, typename ST> __global__ __launch_bounds__(256, 1) void ssm_chunk_f32_kernel(SsmArgs a, Segments sg) {
    extern __shared__ __align__(16) unsigned char lds[];
    const Place at(a, sg, ChunkF<P, S>::HW);
    if (at.skip) return;
    if (at.whole) run_segment_f32<P, S, ST, true>(a, sg, at, lds);
    else run_segment_f32<P, S, ST, false>(a, sg, at, lds);
}

template <int P, int S, typename ST> static hipError_t launch_t(const SsmArgs &a, const Segments &sg, hipStream_t s) {
    using C = ChunkF<P, S>;
    static_assert(C::LDS <= 163840, "LDS");
    const auto kern = ssm_chunk_f32_kernel<P, S, ST>;
    const hipError_t e = hipFuncSetAttribute((const void *)kern, hipFuncAttributeMaxDynamicSharedMemorySize, C::LDS);
    if (e != hipSuccess) return e;
    kern<<<dim3(ssm_units(a, sg) * ssm_head_workgroups(a)), 256, C::LDS, s>>>(a, sg);
    return hipGetLastError();
}
template <int P> static hipError_t launch_s(const SsmArgs &a, const Segments &sg, hipStream_t s) {
    switch (a.s) {
    case 32: return a.state_bf16 ? launch_t<P, 32, bf16>(a, sg, s) : launch_t<P, 32, float>(a, sg, s);
    case 64: return a.state_bf16 ? launch_t<P, 64, bf16>(a, sg, s) : launch_t<P, 64, float>(a, sg, s);
    default: return a.state_bf16 ? launch_t<P, 128, bf16>(a, sg, s) : launch_t<P, 128, float>(a, sg, s);
    }
}
hipError_t launch_ssm_chunk_f32(const SsmArgs &a, const Segments &sg, hipStream_t s) {
    switch (a.p) {
    case 32: return launch_s<32>(a, sg, s);
    case 64: return launch_s<64>(a, sg, s);
    default: return launch_s<128>(a, sg, s);
    }
}

}  // namespace kda
