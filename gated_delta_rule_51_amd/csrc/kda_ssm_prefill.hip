// Selective state-space scan of packed prompts, bf16 io, in chunks of 64
// tokens on the matrix cores.
//
// With G_t the running sum of log-decays within a chunk, S the state before it:
//     M_ts = (C_t . B_s) exp(G_t - G_s) dt_s  (s <= t),  M_tt += D
//     y_t  = exp(G_t) S C_t + sum_s M_ts x_s
//     S'   = exp(G_last) S + sum_s (exp(G_last - G_s) dt_s x_s) B_s^T
// The columns p of a head never mix, so a wave owns 32 of them and keeps its
// part of the state (32 x S) in registers through all chunks of a sequence;
// a workgroup's four waves share one head of 128 columns, two of 64 or four
// of 32 (heads of one group, so B and C are staged once for all).
//
// Operands.  A 32 x 32 x 16 product takes eight consecutive k of a row in a
// lane (k = 8 (lane / 32) + 0..7) and leaves rows 8a + 4 (lane / 32) + b in
// its registers 4a + b.  Rows i of the products over p and n stand for
// column swap23(i) (bits 2 and 3 exchanged), so that a lane's registers hold
// eight consecutive columns: the state then is the next product's operand, and
// y a 16-byte store, without leaving the registers.  M's rows keep their
// order; its k slots are {4h + b, 8 + 4h + b} of every 16 tokens, and the
// transposed reads of x and B take their rows in that order.
//
// Precision.  x, B and C are bf16 and enter exactly.  What is fp32 enters as a
// sum of bf16 terms: M and S in two (remainder 2^-17 of the value, far below
// y's own rounding of 2^-9), dt x exp(.) in three (2^-26), so that the fp32
// states keep fp32's accuracy, in the whole range of bf16.  The sums G are
// formed in fp64 and kept as two floats: differences of large sums would
// otherwise lose the small decays between neighbours.
#include "kda_device.h"
#include "kda_internal.h"
#include "kda_ssm.h"

namespace kda {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ f32x16 mfma(u32x4 a, u32x4 b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

// Four rows of a column: of each 16 lanes, lane l reads 8 bytes (4 columns) of
// row l / 4 and receives column l of the four rows.
__device__ __forceinline__ u32x2 lds_tr(const unsigned char *p) {
    return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                                         (__attribute__((address_space(3))) s16x4 *)(uintptr_t)p));
}

__device__ __forceinline__ float lo_f(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_f(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// v as bf16 terms: t[0] + t[1] (+ t[2]).
template <int TERMS> __device__ __forceinline__ void split(const float (&v)[8], u32x4 (&t)[TERMS]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float x = v[2 * i], y = v[2 * i + 1];
#pragma unroll
        for (int k = 0; k < TERMS; ++k) {
            const uint32_t w = pack_bf16x2(x, y);
            t[k][i] = w;
            if (k + 1 < TERMS) {
                x -= lo_f(w);
                y -= hi_f(w);
            }
        }
    }
}

constexpr int kGateArrays = 5;   // G (two floats), dt, exp(G_last - G) dt, exp(G)

template <int P, int S> struct Chunk {
    static constexpr int WPH = P / 32;          // waves of a head
    static constexpr int HW = 4 / WPH;          // heads of a workgroup
    static constexpr int NT = S / 32;           // 32-wide tiles of the state's columns
    static constexpr int XROW = 256 + 32;       // LDS row strides: 32 bytes past the row keep
    static constexpr int BROW = 2 * S + 32;     // both kinds of reads free of bank conflicts
    static constexpr int PPR = S / 8;           // 16-byte pieces of a row of B
    static constexpr int PB = PPR / 4;          // pieces of B a thread stages
    static constexpr int MBYTES = WPH == 1 ? 0 : 3 * 2 * 2 * 1024;   // M of one head
    static constexpr int OFF_B = 64 * XROW, OFF_C = OFF_B + 64 * BROW, OFF_M = OFF_C + 64 * BROW;
    static constexpr int OFF_G = OFF_M + HW * MBYTES;
    static constexpr int GBYTES = HW * kGateArrays * 256;            // one buffer of gates
    static constexpr int LDS = OFF_G + 2 * GBYTES;
};

// M's tile (rows t of 32 tt, columns s of 32 ss) from the products C_t . B_s,
// as two operands of 16 tokens each in two bf16 terms.
__device__ __forceinline__ void m_tile(const f32x16 &cb, const float *gate, int tt, int ss, int lane, float Dh, u32x4 (&m)[2][2]) {
    const int t = 32 * tt + (lane & 31), hh = lane >> 5;
    const float gt = gate[t], lt = gate[64 + t];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        float v[8];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int s0 = 32 * ss + 8 * (2 * u + k) + 4 * hh;
            const f32x4 gs = *reinterpret_cast<const f32x4 *>(gate + s0), ls = *reinterpret_cast<const f32x4 *>(gate + 64 + s0);
            const f32x4 ds = *reinterpret_cast<const f32x4 *>(gate + 128 + s0);
#pragma unroll
            for (int b = 0; b < 4; ++b) {
                const float e = __builtin_amdgcn_exp2f((gt - gs[b]) + (lt - ls[b])) * ds[b];
                float x = cb[4 * (2 * u + k) + b] * e;
                if (tt == ss) {
                    x = s0 + b == t ? x + Dh : x;
                    x = s0 + b <= t ? x : 0.f;
                }
                v[4 * k + b] = x;
            }
        }
        split<2>(v, m[u]);
    }
}

template <int P, int S, typename ST> __global__ __launch_bounds__(256, 2) void ssm_chunk_kernel(SsmArgs a) {
    using C = Chunk<P, S>;
    extern __shared__ __align__(16) unsigned char lds[];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int hh = lane >> 5, l32 = lane & 31;
    const int hs = wave / C::WPH, pc = wave % C::WPH;   // head of the workgroup, 32-column block of the head

    const int rep = a.heads / a.groups, blocks = (rep + C::HW - 1) / C::HW;
    const int seq = (int)blockIdx.x / (a.groups * blocks), rest = (int)blockIdx.x % (a.groups * blocks);
    const int g = rest / blocks, first = g * rep + rest % blocks * C::HW;   // first head
    const int h = first + hs;
    const bool active = h < (g + 1) * rep;
    const int t0 = a.cu_seqlens[seq], len = a.cu_seqlens[seq + 1] - t0;
    if (len <= 0 && (a.indices || !a.state_out)) return;
    long slot = seq;
    if (a.indices) {
        slot = a.indices[seq];
        if (slot < 0) slot = a.num_slots - 1;
    }

    // state: register 8u + 4k + b of tile nt is column n = 32 nt + 16 u + 8 hh + 4 k + b of row pcol
    const int pcol = (l32 & 0x13) | ((l32 & 4) << 1) | ((l32 & 8) >> 1);
    const long at = ((slot * a.heads + (active ? h : first)) * P + 32 * pc + pcol) * (long)S + 8 * hh;
    f32x16 st[C::NT];
#pragma unroll
    for (int nt = 0; nt < C::NT; ++nt)
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            f32x4 x = {0.f, 0.f, 0.f, 0.f}, y = x;
            if (a.state_in) {
                const ST *p = reinterpret_cast<const ST *>(a.state_in) + at + 32 * nt + 16 * u;
                x = load4(p);
                y = load4(p + 4);
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                st[nt][8 * u + e] = x[e];
                st[nt][8 * u + 4 + e] = y[e];
            }
        }

    // staging of x (16 pieces a row, 16 rows a pass), B and C through registers
    const bf16 *xg = reinterpret_cast<const bf16 *>(a.x) + (long)t0 * a.x_stride + (long)first * P;
    const bf16 *bg = reinterpret_cast<const bf16 *>(a.B) + (long)t0 * a.b_stride + (long)g * S;
    const bf16 *cg = reinterpret_cast<const bf16 *>(a.C) + (long)t0 * a.c_stride + (long)g * S;
    const unsigned xoff = (unsigned)((tid / 16) * a.x_stride + (tid % 16) * 8) * 2;
    const unsigned boff = (unsigned)((tid / C::PPR) * a.b_stride + (tid % C::PPR) * 8) * 2;
    const unsigned coff = (unsigned)((tid / C::PPR) * a.c_stride + (tid % C::PPR) * 8) * 2;
    const bool xin = first + (tid % 16) * 8 / P < (g + 1) * rep;   // the piece's head is there
    u32x4 xr[4], br[C::PB], cr[C::PB];
    auto stage = [&](int c0) {   // rows past the sequence read as zero
        const int rows = min(64, len - c0);
        const __amdgpu_buffer_rsrc_t xs = __builtin_amdgcn_make_buffer_rsrc(
            const_cast<bf16 *>(xg + c0 * a.x_stride), 0, (int)(rows * a.x_stride * 2), kBufferWord3);
        const __amdgpu_buffer_rsrc_t bs = __builtin_amdgcn_make_buffer_rsrc(
            const_cast<bf16 *>(bg + c0 * a.b_stride), 0, (int)(rows * a.b_stride * 2), kBufferWord3);
        const __amdgpu_buffer_rsrc_t cs = __builtin_amdgcn_make_buffer_rsrc(
            const_cast<bf16 *>(cg + c0 * a.c_stride), 0, (int)(rows * a.c_stride * 2), kBufferWord3);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            xr[i] = __builtin_amdgcn_raw_buffer_load_b128(xs, xin ? xoff + (unsigned)(16 * i * a.x_stride * 2) : 0x80000000u, 0, 0);
#pragma unroll
        for (int i = 0; i < C::PB; ++i) {
            br[i] = __builtin_amdgcn_raw_buffer_load_b128(bs, boff + (unsigned)(256 / C::PPR * i * a.b_stride * 2), 0, 0);
            cr[i] = __builtin_amdgcn_raw_buffer_load_b128(cs, coff + (unsigned)(256 / C::PPR * i * a.c_stride * 2), 0, 0);
        }
    };
    auto unstage = [&]() {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            *reinterpret_cast<u32x4 *>(lds + (tid / 16 + 16 * i) * C::XROW + (tid % 16) * 16) = xr[i];
#pragma unroll
        for (int i = 0; i < C::PB; ++i) {
            const int at_l = (tid / C::PPR + 256 / C::PPR * i) * C::BROW + (tid % C::PPR) * 16;
            *reinterpret_cast<u32x4 *>(lds + C::OFF_B + at_l) = br[i];
            *reinterpret_cast<u32x4 *>(lds + C::OFF_C + at_l) = cr[i];
        }
    };

    // gates, by the last wave of each head, a token a lane
    const bool gates = active && pc == C::WPH - 1;
    const double A = gates ? -exp((double)a.A_log[h]) * 1.4426950408889634 : 0.0;
    const float bias = gates && a.dt_bias ? a.dt_bias[h] : 0.f, Dh = active && a.D ? a.D[h] : 0.f;
    const bf16 *dg = reinterpret_cast<const bf16 *>(a.dt) + (long)t0 * a.dt_stride + h;
    float dtv = 0.f;
    auto fetch_dt = [&](int c0) {
        dtv = 0.f;
        if (gates && c0 + lane < len) dtv = io_traits<bf16>::load(dg, (long)(c0 + lane) * a.dt_stride);
    };
    auto make_gates = [&](int c0, int buf) {
        if (!gates) return;
        const float step = c0 + lane < len ? softplus_f(dtv + bias) : 0.f;
        double G = (double)step * A;
#pragma unroll
        for (int m = 1; m < 64; m <<= 1) {
            const double o = __shfl_up(G, m, 64);
            if (lane >= m) G += o;
        }
        const double last = __shfl(G, 63, 64);
        float *q = reinterpret_cast<float *>(lds + C::OFF_G + buf * C::GBYTES) + hs * kGateArrays * 64 + lane;
        const float gh = (float)G;
        q[0] = gh;
        q[64] = (float)(G - (double)gh);
        q[128] = step;
        q[192] = step * __builtin_amdgcn_exp2f((float)(last - G));
        q[256] = __builtin_amdgcn_exp2f(gh);
    };

    if (len > 0) {
        stage(0);
        fetch_dt(0);
        make_gates(0, 0);
    }
    // transposed reads: row (of 4) and column piece of this lane within a 32-column block
    const int trow = 4 * hh + ((lane & 15) >> 2);
    const int tcol = 32 * ((lane >> 4) & 1) + 8 * (((lane & 1) << 1) | ((lane >> 1) & 1));   // bytes
    unsigned char *const mbase = lds + C::OFF_M + hs * C::MBYTES + lane * 16;

    int buf = 0;
    for (int c0 = 0; c0 < len; c0 += 64, buf ^= 1) {
        unstage();
        __syncthreads();
        const float *gate = reinterpret_cast<const float *>(lds + C::OFF_G + buf * C::GBYTES) + hs * kGateArrays * 64;
        // z of this chunk (used last) and the next chunk's rows: in flight meanwhile
        u32x4 zr[2][2];
        if (a.z) {
#pragma unroll
            for (int tt = 0; tt < 2; ++tt) {
                const int t = c0 + 32 * tt + l32;
                const bf16 *zp = reinterpret_cast<const bf16 *>(a.z) + (long)(t0 + min(t, len - 1)) * a.z_stride +
                                 (long)(active ? h : first) * P + 32 * pc + 8 * hh;
                zr[tt][0] = *reinterpret_cast<const u32x4 *>(zp);
                zr[tt][1] = *reinterpret_cast<const u32x4 *>(zp + 16);
            }
        }
        const bool more = c0 + 64 < len;
        if (more) {
            stage(c0 + 64);
            fetch_dt(c0 + 64);
        }

        // C_t . B_s, and M from it: tiles (t, s) = (0, 0), (1, 0), (1, 1) shared by the head's waves
        u32x4 m[C::WPH == 1 ? 3 : 1][2][2];
        if (active) {
#pragma unroll
            for (int tile = 0; tile < 3; ++tile) {
                const int owner = C::WPH == 4 ? tile : C::WPH == 2 ? tile & 1 : 0;
                if (owner != pc) continue;
                const int tt = tile > 0, ss = tile > 1;
                f32x16 acc;
#pragma unroll
                for (int i = 0; i < 16; ++i) acc[i] = 0.f;
#pragma unroll
                for (int u = 0; u < S / 16; ++u) {
                    const u32x4 bo = *reinterpret_cast<const u32x4 *>(lds + C::OFF_B + (32 * ss + l32) * C::BROW + 32 * u + 16 * hh);
                    const u32x4 co = *reinterpret_cast<const u32x4 *>(lds + C::OFF_C + (32 * tt + l32) * C::BROW + 32 * u + 16 * hh);
                    acc = mfma(bo, co, acc);
                }
                constexpr bool own = C::WPH == 1;
                u32x4(&mt)[2][2] = m[own ? tile : 0];
                m_tile(acc, gate, tt, ss, lane, Dh, mt);
                if constexpr (!own) {
#pragma unroll
                    for (int u = 0; u < 2; ++u)
#pragma unroll
                        for (int k = 0; k < 2; ++k) *reinterpret_cast<u32x4 *>(mbase + (tile * 4 + u * 2 + k) * 1024) = mt[u][k];
                }
            }
            if (more) make_gates(c0 + 64, buf ^ 1);
        }

        // y = exp(G) S C
        f32x16 y[2];
#pragma unroll
        for (int i = 0; i < 16; ++i) y[0][i] = y[1][i] = 0.f;
#pragma unroll
        for (int nt = 0; nt < C::NT; ++nt)
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                float v[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] = st[nt][8 * u + e];
                u32x4 s[2];
                split<2>(v, s);
#pragma unroll
                for (int tt = 0; tt < 2; ++tt) {
                    const u32x4 co = *reinterpret_cast<const u32x4 *>(lds + C::OFF_C + (32 * tt + l32) * C::BROW + 64 * nt + 32 * u + 16 * hh);
                    y[tt] = mfma(s[0], co, y[tt]);
                    y[tt] = mfma(s[1], co, y[tt]);
                }
            }
#pragma unroll
        for (int tt = 0; tt < 2; ++tt) {
            const float e = gate[256 + 32 * tt + l32];
#pragma unroll
            for (int i = 0; i < 16; ++i) y[tt][i] *= e;
        }
        const float all = gate[256 + 63];
#pragma unroll
        for (int nt = 0; nt < C::NT; ++nt)
#pragma unroll
            for (int i = 0; i < 16; ++i) st[nt][i] *= all;
        if constexpr (C::WPH > 1) __syncthreads();

        // y += M x;  S += (weights x) B^T, 16 tokens at a time
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int ss = k >> 1, u = k & 1;
            const int row = 16 * k + trow;
            const unsigned char *xp = lds + row * C::XROW + 64 * wave + tcol;
            const u32x2 x0 = lds_tr(xp), x1 = lds_tr(xp + 8 * C::XROW);
            const u32x4 xo = {x0[0], x0[1], x1[0], x1[1]};
#pragma unroll
            for (int tt = ss; tt < 2; ++tt) {
                const int tile = tt + ss;
                u32x4 m0, m1;
                if constexpr (C::WPH == 1) {
                    m0 = m[tile][u][0];
                    m1 = m[tile][u][1];
                } else {
                    m0 = *reinterpret_cast<const u32x4 *>(mbase + (tile * 4 + u * 2) * 1024);
                    m1 = *reinterpret_cast<const u32x4 *>(mbase + (tile * 4 + u * 2 + 1) * 1024);
                }
                y[tt] = mfma(xo, m0, y[tt]);
                y[tt] = mfma(xo, m1, y[tt]);
            }
            const f32x4 w0 = *reinterpret_cast<const f32x4 *>(gate + 192 + 16 * k + 4 * hh);
            const f32x4 w1 = *reinterpret_cast<const f32x4 *>(gate + 192 + 16 * k + 8 + 4 * hh);
            float v[8];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                v[2 * e] = lo_f(xo[e]) * w0[2 * e];
                v[2 * e + 1] = hi_f(xo[e]) * w0[2 * e + 1];
                v[4 + 2 * e] = lo_f(xo[2 + e]) * w1[2 * e];
                v[5 + 2 * e] = hi_f(xo[2 + e]) * w1[2 * e + 1];
            }
            u32x4 wx[3];
            split<3>(v, wx);
#pragma unroll
            for (int nt = 0; nt < C::NT; ++nt) {
                const unsigned char *bp = lds + C::OFF_B + row * C::BROW + 64 * nt + tcol;
                const u32x2 b0 = lds_tr(bp), b1 = lds_tr(bp + 8 * C::BROW);
                const u32x4 bo = {b0[0], b0[1], b1[0], b1[1]};
#pragma unroll
                for (int j = 0; j < 3; ++j) st[nt] = mfma(bo, wx[j], st[nt]);
            }
        }

        if (active) {
#pragma unroll
            for (int tt = 0; tt < 2; ++tt) {
                const int t = c0 + 32 * tt + l32;
                if (a.z) {
#pragma unroll
                    for (int u = 0; u < 2; ++u)
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float z0 = lo_f(zr[tt][u][i]), z1 = hi_f(zr[tt][u][i]);
                            y[tt][8 * u + 2 * i] *= z0 * sigmoid_f(z0);
                            y[tt][8 * u + 2 * i + 1] *= z1 * sigmoid_f(z1);
                        }
                }
                if (t < len) {
                    bf16 *yp = reinterpret_cast<bf16 *>(a.y) + ((long)(t0 + t) * a.heads + h) * P + 32 * pc + 8 * hh;
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        u32x4 w;
#pragma unroll
                        for (int i = 0; i < 4; ++i) w[i] = pack_bf16x2(y[tt][8 * u + 2 * i], y[tt][8 * u + 2 * i + 1]);
                        *reinterpret_cast<u32x4 *>(yp + 16 * u) = w;
                    }
                }
            }
        }
        __syncthreads();   // every wave has read this chunk
    }

    if (a.state_out && active) {
#pragma unroll
        for (int nt = 0; nt < C::NT; ++nt)
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                ST *p = reinterpret_cast<ST *>(a.state_out) + at + 32 * nt + 16 * u;
                if constexpr (sizeof(ST) == 4) {
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const f32x4 x = {st[nt][8 * u + 4 * k], st[nt][8 * u + 4 * k + 1], st[nt][8 * u + 4 * k + 2],
                                         st[nt][8 * u + 4 * k + 3]};
                        *reinterpret_cast<f32x4 *>(p + 4 * k) = x;
                    }
                } else {
                    u32x4 w;
#pragma unroll
                    for (int i = 0; i < 4; ++i) w[i] = pack_bf16x2(st[nt][8 * u + 2 * i], st[nt][8 * u + 2 * i + 1]);
                    *reinterpret_cast<u32x4 *>(p) = w;
                }
            }
    }
}

template <int P, int S, typename ST> static hipError_t launch_chunk(const SsmArgs &a, hipStream_t stream) {
    using C = Chunk<P, S>;
    static_assert(C::LDS <= 163840, "LDS");
    const int rep = a.heads / a.groups;
    const dim3 grid(a.num_seqs * a.groups * ((rep + C::HW - 1) / C::HW));
    ssm_chunk_kernel<P, S, ST><<<grid, 256, C::LDS, stream>>>(a);
    return hipGetLastError();
}
template <int P, int S> static hipError_t launch_st(const SsmArgs &a, hipStream_t s) {
    return a.state_bf16 ? launch_chunk<P, S, bf16>(a, s) : launch_chunk<P, S, float>(a, s);
}
template <int P> static hipError_t launch_s(const SsmArgs &a, hipStream_t s) {
    switch (a.s) {
    case 32: return launch_st<P, 32>(a, s);
    case 64: return launch_st<P, 64>(a, s);
    default: return launch_st<P, 128>(a, s);
    }
}

size_t ssm_prefill_workspace_bytes(int, int, int, int, int, bool) { return 0; }

hipError_t launch_ssm_prefill(const SsmArgs &a, void *, hipStream_t s) {
    if (!a.io_bf16) return launch_ssm_run(a, s);
    switch (a.p) {
    case 32: return launch_s<32>(a, s);
    case 64: return launch_s<64>(a, s);
    default: return launch_s<128>(a, s);
    }
}

}  // namespace kda
