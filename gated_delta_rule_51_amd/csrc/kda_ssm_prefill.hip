// Selective state-space scan of packed prompts (bf16 io; the launches of both
// kinds), in chunks of 64 tokens on the matrix cores.
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
// Precision.  x, B and C are bf16 and enter exactly.  What is fp32 (M, S and
// dt x exp(.)) enters as the sum of three bf16 terms, which hold all its 24
// bits, so y and the states keep fp32's accuracy, also where large parts of a
// state cancel in S C or of M in M x; two terms (17 bits) lost y there, and
// elsewhere changed y's last bit four times as often.  They took 349 and 278 us
// for the two workloads below in a run where three take 390 and 294.  The sums
// G are formed in fp64 and kept as two floats: differences of large sums would
// otherwise lose the small decays between neighbours.
//
// Segments.  A chain of chunks is latency bound, and few long sequences leave
// the chip idle, so sequences are cut into segments.  The first launch runs
// every sequence's first segment whole and the states alone of those between
// the first and the last, from zero; a second carries the states across them
// (state = decay of the segment x the state before it + its own); the last runs
// the other segments whole, each from the state before it.  Sequences of one or
// two segments thus do no work twice.
//
// What bounds it.  At P = S = 128 a wave's chunk takes 122 products of 32
// cycles and about 1200 vector instructions of 4, two waves a SIMD, most of them
// the splitting of fp32 operands, the gating by z and M's exponentials, so the
// vector units set the pace: they issue in 51 to 60% of the busy CUs' cycles, the
// matrix cores are busy in 41 to 36%, and the tails of two launches leave 17 to
// 27% of the CUs without work.  Memory is at 1.8 TB/s.  16 prompts of 512 to 4096
// tokens x 32 heads x (128 x 128): 375 to 400 us by the run (0.69 GB, 64 GFLOP);
// one of 32,768 x 32 heads x (64 x 128), gated: 287 to 295 us, of which the first
// launch takes about 95 and the carry 22.  Held back by registers: P = S = 128
// spills 20, P = 32 with S = 128 55.
#include <algorithm>
#include <type_traits>

#include "kda_ssm_chunk.h"

namespace kda {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ f32x16 mfma(u32x4 a, u32x4 b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

// Four rows of a column: of each 16 lanes, lane l reads 8 bytes (4 columns) of
// row l / 4 and receives column l of the four rows.
__device__ __forceinline__ u32x2 lds_tr(uint32_t at) {
    return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4 *)(uintptr_t)at));
}
__device__ __forceinline__ u32x4 lds_row(uint32_t at) {
    return *(const __attribute__((address_space(3))) u32x4 *)(uintptr_t)at;
}

__device__ __forceinline__ float lo_f(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_f(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// Two floats as words of three bf16 terms each, t[0] + t[1] + t[2], exactly: a
// term is cut off after 8 bits, not rounded, so three hold the 24 and the first
// never passes the value (rounded, one above bf16's largest became infinite).
constexpr int kTerms = 3;
__device__ __forceinline__ void split2(float x, float y, uint32_t (&t)[kTerms]) {
#pragma unroll
    for (int k = 0; k < kTerms; ++k) {
        t[k] = __builtin_amdgcn_perm(__float_as_uint(y), __float_as_uint(x), 0x07060302);   // both upper halves
        x -= __uint_as_float(__float_as_uint(x) & 0xffff0000u);
        y -= __uint_as_float(__float_as_uint(y) & 0xffff0000u);
    }
}
__device__ __forceinline__ void split(const float (&v)[8], u32x4 (&t)[kTerms]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t w[kTerms];
        split2(v[2 * i], v[2 * i + 1], w);
#pragma unroll
        for (int k = 0; k < kTerms; ++k) t[k][i] = w[k];
    }
}

template <int P, int S> struct Chunk {
    static constexpr int WPH = P / 32;          // waves of a head
    static constexpr int HW = 4 / WPH;          // heads of a workgroup
    static constexpr int NT = S / 32;           // 32-wide tiles of the state's columns
    static constexpr int PPR = S / 8;           // 16-byte pieces of a row of B
    static constexpr int PB = PPR / 4;          // pieces of B a thread stages
    static constexpr int OFF_B = 64 * 256, OFF_C = OFF_B + 64 * 2 * S, OFF_M = OFF_C + 64 * 2 * S;
    static constexpr int GBYTES = HW * kGateArrays * 256;            // one buffer of gates
    // M of a head, three tiles: as terms, each formed once, or as floats that every
    // wave of the head splits, where terms would leave no room for two workgroups
    static constexpr int TERM_BYTES = 3 * 2 * kTerms * 1024;
    static constexpr bool MTERMS = WPH > 1 && OFF_M + HW * TERM_BYTES + 2 * GBYTES <= 81920;
    static constexpr int MBYTES = WPH == 1 ? 0 : MTERMS ? TERM_BYTES : 3 * 4096;
    static constexpr int OFF_G = OFF_M + HW * MBYTES;
    static constexpr int LDS = OFF_G + 2 * GBYTES;
};

// Byte offset of a row's 16-byte piece in an LDS tile of PPR pieces a row.
// Pieces are exchanged within rows so that neither 16 rows of one piece (the
// operands' own order) nor four rows of two neighbours (the transposed reads)
// meet in a bank.
template <int PPR> __device__ __forceinline__ int swizzle(int row) {
    const int q2 = row / (16 / PPR) * 2;
    return (q2 & (PPR - 1)) | ((q2 / PPR) & 1);
}
template <int PPR> __device__ __forceinline__ int tile_at(int row, int piece) {
    return row * PPR * 16 + ((piece ^ swizzle<PPR>(row & 15)) << 4);   // repeats every 16 rows
}

// A workgroup's segment; without Y its state alone.
template <int P, int S, typename ST, bool Y>
__device__ __forceinline__ void run_segment(const SsmArgs &a, const Segments &sg, const Place &at, unsigned char *lds) {
    using C = Chunk<P, S>;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int hs = wave / C::WPH, pc = wave % C::WPH;   // head of the workgroup, 32-column block of the head

    const int g = at.g, first = at.first, h = first + hs, t0 = at.t0, len = at.len;
    const bool active = h < at.last;

    // state: register 8u + 4k + b of tile nt is column n = 32 nt + 16 u + 8 hh + 4 k + b of row pcol
    const auto in_heads = [&](int l) {
        const int pcol = (l & 0x13) | ((l & 4) << 1) | ((l & 8) >> 1);
        return (long)((active ? h : first) * P + 32 * pc + pcol) * S + 8 * (l >> 5);
    };
    const long one = (long)a.heads * P * S;
    f32x16 st[C::NT];
    const long in_head = in_heads(lane);
#pragma unroll
    for (int nt = 0; nt < C::NT; ++nt)
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            f32x4 x = {0.f, 0.f, 0.f, 0.f}, y = x;
            if (sg.later) {
                const float *p = sg.states + (at.place - 1) * one + in_head + 32 * nt + 16 * u;
                x = load4(p);
                y = load4(p + 4);
            } else if (a.state_in && at.local == 0) {
                const ST *p = reinterpret_cast<const ST *>(a.state_in) + at.row * one + in_head + 32 * nt + 16 * u;
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
    // z and y: row l32 of 32, the wave's columns
    const bf16 *yg = uniform(reinterpret_cast<const bf16 *>(a.y) + (long)t0 * a.heads * P + (long)h * P + 32 * pc);
    const bf16 *zg = uniform(reinterpret_cast<const bf16 *>(a.z) + (long)t0 * a.z_stride + (long)(active ? h : first) * P + 32 * pc);
    u32x4 xr[4], br[C::PB], cr[C::PB];
    // `each` rows from row `from`; rows past the sequence read as zero
    auto rows_at = [&](const bf16 *base, long stride, int from, int each) {
        // (clamped on the vector unit, whose result would make the load loop over descriptors)
        const int rows = __builtin_amdgcn_readfirstlane(max(0, min(each, len - from)));
        return __builtin_amdgcn_make_buffer_rsrc(const_cast<bf16 *>(base + from * stride), 0, (int)(rows * stride * 2), kBufferWord3);
    };
    // A burst of loads stalls the wave until the caches take them, so they are
    // issued a few at a time: part q of 4 of x, of B, of C.
    auto stage_x = [&](int c0, int lane, int q) {
        const int tid = 64 * wave + lane;
        const unsigned off = (unsigned)((tid / 16) * (int)a.x_stride + (tid % 16) * 8) * 2;
        const bool in = first + (tid % 16) * 8 / P < at.last;   // the piece's head is there
        xr[q] = __builtin_amdgcn_raw_buffer_load_b128(rows_at(xg, a.x_stride, c0 + 16 * q, 16), in ? off : 0x80000000u, 0, 0);
    };
    constexpr int each = 256 / C::PPR;   // rows of B and C a pass of the workgroup loads
    auto stage_b = [&](int c0, int lane, int q) {
        const int tid = 64 * wave + lane;
        if (q < C::PB)
            br[q] = __builtin_amdgcn_raw_buffer_load_b128(rows_at(bg, a.b_stride, c0 + each * q, each),
                                                          (unsigned)((tid / C::PPR) * (int)a.b_stride + (tid % C::PPR) * 8) * 2, 0, 0);
    };
    auto stage_c = [&](int c0, int lane, int q) {
        const int tid = 64 * wave + lane;
        if (Y && q < C::PB)
            cr[q] = __builtin_amdgcn_raw_buffer_load_b128(rows_at(cg, a.c_stride, c0 + each * q, each),
                                                          (unsigned)((tid / C::PPR) * (int)a.c_stride + (tid % C::PPR) * 8) * 2, 0, 0);
    };
    auto unstage_xb = [&](int lane) {
        const int tid = 64 * wave + lane;
#pragma unroll
        for (int i = 0; i < 4; ++i) *reinterpret_cast<u32x4 *>(lds + tile_at<16>(tid / 16 + 16 * i, tid % 16)) = xr[i];
#pragma unroll
        for (int i = 0; i < C::PB; ++i)
            *reinterpret_cast<u32x4 *>(lds + C::OFF_B + tile_at<C::PPR>(tid / C::PPR + each * i, tid % C::PPR)) = br[i];
    };
    auto unstage_c = [&](int lane) {
        const int tid = 64 * wave + lane;
#pragma unroll
        for (int i = 0; i < C::PB; ++i)
            *reinterpret_cast<u32x4 *>(lds + C::OFF_C + tile_at<C::PPR>(tid / C::PPR + each * i, tid % C::PPR)) = cr[i];
    };

    // gates, by the last wave of each head, a token a lane; an empty sequence has
    // none, and without any token A_log may be NULL
    const bool gates = active && len > 0 && pc == C::WPH - 1;
    const double A = uniform(gates ? -exp((double)a.A_log[h]) * 1.4426950408889634 : 0.0);
    const float bias = gates && a.dt_bias ? a.dt_bias[h] : 0.f, Dh = active && a.D ? a.D[h] : 0.f;
    const bf16 *dg = reinterpret_cast<const bf16 *>(a.dt) + (long)t0 * a.dt_stride + h;
    uint32_t dtv = 0;       // bits, of a chunk ahead: converted when they are used
    double through = 0.0;   // log2 of the segment's decay
    auto fetch_dt = [&](int c0, int lane) {
        dtv = reinterpret_cast<const uint16_t *>(dg)[(long)min(c0 + lane, len - 1) * a.dt_stride];
    };
    auto make_gates = [&](int c0, int buf, int lane) {
        const float step = c0 + lane < len ? softplus_f(lo_f(dtv) + bias) : 0.f;
        float *q = reinterpret_cast<float *>(lds + C::OFF_G + buf * C::GBYTES) + hs * kGateArrays * 64 + lane;
        through = uniform(through + write_gates(q, step, A));
    };

    if (len > 0) {
        if (gates) {
            fetch_dt(0, lane);
            make_gates(0, 0, lane);
            fetch_dt(64, lane);   // a chunk ahead of its use: memory answers in order, and the rows' loads are slower
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            stage_x(0, lane, q);
            stage_b(0, lane, q);
            stage_c(0, lane, q);
        }
        if constexpr (Y && C::WPH > 1) unstage_c(lane);
    }
    int buf = 0;
    const int lane0 = lane;
    for (int c0 = 0; c0 < len; c0 += 64, buf ^= 1) {
        // What depends on the lane is formed anew in every chunk: kept through
        // the loop it takes some 40 registers, and what is spilled for them
        // waits, when it is read back, for the rows on their way.
        int lane = lane0;
        asm volatile("" : "+v"(lane));
        lane &= 63;
        const int hh = lane >> 5, l32 = lane & 31;
        // transposed reads: row (of 4) and column piece (8 bytes) of this lane within a 32-column block
        const int trow = 4 * hh + ((lane & 15) >> 2), tpiece = 2 * ((lane >> 4) & 1) + (lane & 1), thalf = (lane & 2) << 2;
        // LDS addresses of the operands: another piece of a row is an exclusive or
        // away (one instruction; formed from rows and pieces they took five), other
        // rows and tiles a constant
        const uint32_t lds0 = (uint32_t)(uintptr_t)lds;
        const uint32_t row_at = lds0 + tile_at<C::PPR>(l32, hh);
        const uint32_t x_at[2] = {lds0 + tile_at<16>(trow, 4 * wave + tpiece) + thalf, lds0 + tile_at<16>(trow + 8, 4 * wave + tpiece) + thalf};
        const uint32_t b_at[2] = {lds0 + tile_at<C::PPR>(trow, tpiece) + thalf, lds0 + tile_at<C::PPR>(trow + 8, tpiece) + thalf};
        const auto operand_row = [&](int part, int rows, int u) {   // rows of 32 of B or C, pieces 2u and 2u + 1
            return lds_row((row_at ^ (u << 5)) + part + rows * 32 * C::PPR * 16);
        };
        unsigned char *const mbase = lds + C::OFF_M + hs * C::MBYTES + lane * 16;
        unstage_xb(lane);
        if constexpr (Y && C::WPH == 1) unstage_c(lane);
        __syncthreads();
        const float *gate = reinterpret_cast<const float *>(lds + C::OFF_G + buf * C::GBYTES) + hs * kGateArrays * 64;
        const bool more = c0 + 64 < len;
        // The next chunk's C is loaded here and takes this one's place after the
        // barrier below; x and B are loaded after that one, for the loop's head.
        // (Past the end there are no rows and the loads return zeros: no branch.)
#pragma unroll
        for (int q = 0; q < 4; ++q) stage_c(c0 + 64, lane, q);

        // C_t . B_s: tiles (t, s) = (0, 0), (1, 0), (1, 1), shared by the waves of
        // a head; a head's only wave forms them where it uses them
        auto products = [&](int tt, int ss) {
            f32x16 acc;
#pragma unroll
            for (int i = 0; i < 16; ++i) acc[i] = 0.f;
#pragma unroll
            for (int u = 0; u < S / 16; ++u) {
                acc = mfma(operand_row(C::OFF_B, ss, u), operand_row(C::OFF_C, tt, u), acc);
            }
            return acc;
        };
        auto form_m = [&](int tt, int ss, float(&mt)[2][8]) {
            const f32x16 cb = products(tt, ss);
            const float gt = gate[32 * tt + l32], lt = gate[64 + 32 * tt + l32];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                float v[4];
                m_part(cb, gate, tt, ss, q, lane, Dh, gt, lt, v);
#pragma unroll
                for (int b = 0; b < 4; ++b) mt[q / 2][4 * (q % 2) + b] = v[b];
            }
        };
        float m[2][2][8];
        if (gates && more) {
            make_gates(c0 + 64, buf ^ 1, lane);
            fetch_dt(c0 + 128, lane);
        }

        // y = exp(G) S C, and under these products the arithmetic of M's tiles
        // tile0 .. tile0 + TILES - 1
        f32x16 y[2];
        auto from_state = [&](auto count, int tile0) {
            constexpr int TILES = decltype(count)::value, NS = S / 16;
            f32x16 cb[TILES > 0 ? TILES : 1];
            float gt[TILES > 0 ? TILES : 1], lt[TILES > 0 ? TILES : 1], mv[8];
#pragma unroll
            for (int j = 0; j < TILES; ++j) {
                const int tt = tile0 + j > 0;
                cb[j] = products(tt, tile0 + j > 1);
                gt[j] = gate[32 * tt + l32];
                lt[j] = gate[64 + 32 * tt + l32];
            }
#pragma unroll
            for (int i = 0; i < 16; ++i) y[0][i] = y[1][i] = 0.f;
            u32x4 co[2];   // C's operand of one step ahead
#pragma unroll
            for (int tt = 0; tt < 2; ++tt)
                co[tt] = operand_row(C::OFF_C, tt, 0);
#pragma unroll
            for (int i = 0; i < NS; ++i) {
                u32x4 cn[2];
                if (i + 1 < NS) {
#pragma unroll
                    for (int tt = 0; tt < 2; ++tt)
                        cn[tt] = operand_row(C::OFF_C, tt, i + 1);
                }
                float v[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] = st[i / 2][8 * (i % 2) + e];
                u32x4 s[kTerms];
                split(v, s);
#pragma unroll
                for (int j = 0; j < kTerms; ++j)
#pragma unroll
                    for (int tt = 0; tt < 2; ++tt) y[tt] = mfma(s[j], co[tt], y[tt]);
#pragma unroll
                for (int part = i * 4 * TILES / NS; part < (i + 1) * 4 * TILES / NS; ++part) {
                    const int j = part / 4, q = part % 4, tile = tile0 + j;
                    float v4[4];
                    m_part(cb[j], gate, tile > 0, tile > 1, q, lane, Dh, gt[j], lt[j], v4);
#pragma unroll
                    for (int b = 0; b < 4; ++b) mv[4 * (q % 2) + b] = v4[b];
                    if (C::MTERMS && q % 2) {
                        u32x4 mt[kTerms];
                        split(mv, mt);
#pragma unroll
                        for (int k = 0; k < kTerms; ++k)
                            *reinterpret_cast<u32x4 *>(mbase + ((tile * 2 + q / 2) * kTerms + k) * 1024) = mt[k];
                    } else if (!C::MTERMS) {
                        *reinterpret_cast<f32x4 *>(mbase + (tile * 4 + q) * 1024) = f32x4{v4[0], v4[1], v4[2], v4[3]};
                    }
                }
#pragma unroll
                for (int j = 0; j < 2 * kTerms; ++j) {   // a product, then arithmetic that runs under it
                    __builtin_amdgcn_sched_group_barrier(0x8, 1, 0);
                    __builtin_amdgcn_sched_group_barrier(0x2, TILES == 0 ? 10 : 14, 0);
                }
                co[0] = cn[0];
                co[1] = cn[1];
            }
#pragma unroll
            for (int tt = 0; tt < 2; ++tt) {
                const float e = gate[256 + 32 * tt + l32];
#pragma unroll
                for (int i = 0; i < 16; ++i) y[tt][i] *= e;
            }
        };
        if constexpr (Y) {
            using std::integral_constant;
            // tiles of M by wave: 0, 1, 2 and none, or 0, 1 and 2 (the last wave has the gates)
            if (C::WPH == 4 && active && pc < 3) from_state(integral_constant<int, 1>{}, pc);
            else if (C::WPH == 2 && active && pc == 0) from_state(integral_constant<int, 2>{}, 0);
            else if (C::WPH == 2 && active) from_state(integral_constant<int, 1>{}, 2);
            else from_state(integral_constant<int, 0>{}, 0);
        }
        const float all = gate[256 + 63];
        if constexpr (Y && C::WPH > 1) __syncthreads();   // M is there; C is no longer needed
        __builtin_amdgcn_sched_barrier(0);

        // y += M x;  S += (weights x) B^T, 16 tokens at a time, B's operands two
        // products ahead, with the next chunk's rows loaded in between
        u32x4 zr[2][2], xo, bo[3], mo[2][C::MTERMS ? kTerms : 2];
        f32x4 w[2];
        auto operand_x = [&](int k) {
            const u32x2 x0 = lds_tr(x_at[0] + k * 16 * 256), x1 = lds_tr(x_at[1] + k * 16 * 256);
            return u32x4{x0[0], x0[1], x1[0], x1[1]};
        };
        auto operand_b = [&](int step) {
            const int nt = step % C::NT, part = C::OFF_B + step / C::NT * 16 * C::PPR * 16;
            const u32x2 b0 = lds_tr((b_at[0] ^ (nt << 6)) + part), b1 = lds_tr((b_at[1] ^ (nt << 6)) + part);
            return u32x4{b0[0], b0[1], b1[0], b1[1]};
        };
        auto operands_m = [&](int k) {
            if constexpr (Y && C::WPH > 1) {
                constexpr int each = C::MTERMS ? kTerms : 2;
#pragma unroll
                for (int tt = k >> 1; tt < 2; ++tt)
#pragma unroll
                    for (int j = 0; j < each; ++j)
                        mo[tt][j] = *reinterpret_cast<const u32x4 *>(mbase + (((tt + (k >> 1)) * 2 + (k & 1)) * each + j) * 1024);
            }
        };
        auto weights = [&](int k) {
            w[0] = *reinterpret_cast<const f32x4 *>(gate + 192 + 16 * k + 4 * hh);
            w[1] = *reinterpret_cast<const f32x4 *>(gate + 192 + 16 * k + 8 + 4 * hh);
        };
        // words e of the three terms of weight x x
        u32x4 wx[kTerms];
        auto weigh = [&](int e) {
            uint32_t t[kTerms];
            split2(lo_f(xo[e]) * w[e / 2][2 * e % 4], hi_f(xo[e]) * w[e / 2][(2 * e + 1) % 4], t);
#pragma unroll
            for (int j = 0; j < kTerms; ++j) wx[j][e] = t[j];
        };
        xo = operand_x(0);
        operands_m(0);
        weights(0);
        bo[0] = operand_b(0);
        bo[1] = operand_b(1);
        // (a head's only wave still forms M from C below: its workgroup waits for the loop's head)
        if constexpr (Y && C::WPH > 1) unstage_c(lane);
#pragma unroll
        for (int e = 0; e < 4; ++e) weigh(e);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int ss = k >> 1, u = k & 1;
            stage_x(c0 + 64, lane, k);
            stage_b(c0 + 64, lane, k);
            if (Y && k == 2 && a.z) {   // z of this chunk
                const unsigned zoff = (unsigned)(l32 * (int)a.z_stride + 8 * hh) * 2;
#pragma unroll
                for (int tt = 0; tt < 2; ++tt) {
                    const __amdgpu_buffer_rsrc_t zs = rows_at(zg, a.z_stride, c0 + 32 * tt, 32);
                    zr[tt][0] = __builtin_amdgcn_raw_buffer_load_b128(zs, zoff, 0, 0);
                    zr[tt][1] = __builtin_amdgcn_raw_buffer_load_b128(zs, zoff + 32, 0, 0);
                }
            }
            if constexpr (Y && C::WPH == 1) {
                if (u == 0) {
#pragma unroll
                    for (int tt = ss; tt < 2; ++tt) form_m(tt, ss, m[tt]);
                }
            }
            if constexpr (Y) {
                u32x4 mt[2][kTerms];
#pragma unroll
                for (int tt = ss; tt < 2; ++tt) {
                    if constexpr (C::MTERMS) {
#pragma unroll
                        for (int j = 0; j < kTerms; ++j) mt[tt][j] = mo[tt][j];
                    } else if constexpr (C::WPH == 1) {
                        split(m[tt][u], mt[tt]);
                    } else {
                        float v[8];
#pragma unroll
                        for (int e = 0; e < 8; ++e) v[e] = __uint_as_float(mo[tt][e / 4][e % 4]);
                        split(v, mt[tt]);
                    }
                }
#pragma unroll
                for (int j = 0; j < kTerms; ++j)
#pragma unroll
                    for (int tt = ss; tt < 2; ++tt) y[tt] = mfma(xo, mt[tt][j], y[tt]);
            }
            // The next 16 tokens' weighted x is split between this one's products,
            // and the state decays just before its first.
            const u32x4 w0 = wx[0], w1 = wx[1], w2 = wx[2];
#pragma unroll
            for (int nt = 0; nt < C::NT; ++nt) {
                const int step = k * C::NT + nt;
                if (step + 2 < 4 * C::NT) bo[(step + 2) % 3] = operand_b(step + 2);
                if (nt == 0 && k < 3) {
                    xo = operand_x(k + 1);
                    weights(k + 1);
                    operands_m(k + 1);
                }
                __builtin_amdgcn_sched_barrier(0);   // each product keeps the arithmetic that runs under it
                if (k == 0) {
#pragma unroll
                    for (int i = 0; i < 16; ++i) st[nt][i] *= all;
                }
                st[nt] = mfma(bo[step % 3], w0, st[nt]);
                st[nt] = mfma(bo[step % 3], w1, st[nt]);
                st[nt] = mfma(bo[step % 3], w2, st[nt]);
                if (k < 3) {
#pragma unroll
                    for (int e = nt * 4 / C::NT; e < (nt + 1) * 4 / C::NT; ++e) weigh(e);
                }
            }
        }

        if (Y && active) {
            const unsigned yoff = (unsigned)(l32 * a.heads * P + 8 * hh) * 2;
#pragma unroll
            for (int tt = 0; tt < 2; ++tt) {
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
                const __amdgpu_buffer_rsrc_t ys = rows_at(yg, (long)a.heads * P, c0 + 32 * tt, 32);
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    u32x4 w;
#pragma unroll
                    for (int i = 0; i < 4; ++i) w[i] = pack2(y[tt][8 * u + 2 * i], y[tt][8 * u + 2 * i + 1]);
                    __builtin_amdgcn_raw_buffer_store_b128(w, ys, yoff + 32 * u, 0, 0);
                }
            }
        }
        __syncthreads();   // every wave has read this chunk
    }

    const bool last = at.local == at.segs - 1;   // else the state goes to the segment's place
    if (!active || (last ? !a.state_out : sg.later)) return;
    if (!last && gates && lane == 0) sg.decays[(long)at.place * a.heads + h] = __builtin_amdgcn_exp2f((float)through);
    int again = lane;   // the offsets formed anew, not kept through the loop
    asm volatile("" : "+v"(again));
    const long out_head = in_heads(again);
#pragma unroll
    for (int nt = 0; nt < C::NT; ++nt)
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            f32x4 x[2];
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e / 4][e % 4] = st[nt][8 * u + e];
            if (!last) {
                float *p = sg.states + at.place * one + out_head + 32 * nt + 16 * u;
                *reinterpret_cast<f32x4 *>(p) = x[0];
                *reinterpret_cast<f32x4 *>(p + 4) = x[1];
                continue;
            }
            ST *p = reinterpret_cast<ST *>(a.state_out) + at.row * one + out_head + 32 * nt + 16 * u;
            if constexpr (sizeof(ST) == 4) {
                *reinterpret_cast<f32x4 *>(p) = x[0];
                *reinterpret_cast<f32x4 *>(p + 4) = x[1];
            } else {
                const u32x4 w = {pack2(x[0][0], x[0][1]), pack2(x[0][2], x[0][3]), pack2(x[1][0], x[1][1]), pack2(x[1][2], x[1][3])};
                *reinterpret_cast<u32x4 *>(p) = w;
            }
        }
}

template <int P, int S, typename ST> __global__ __launch_bounds__(256, 2) void ssm_chunk_kernel(SsmArgs a, Segments sg) {
    extern __shared__ __align__(1024) unsigned char lds[];   // rows of pieces start on 256 bytes
    const Place at(a, sg, Chunk<P, S>::HW);
    if (at.skip) return;
    if (at.whole) run_segment<P, S, ST, true>(a, sg, at, lds);
    else run_segment<P, S, ST, false>(a, sg, at, lds);
}

// Segments loaded at once, as their loads do not wait for the sums: one prompt
// of 32,768 tokens (62 states of 1 MB) 28 -> 23 us, 5.7 TB/s of reads and writes.
constexpr int kCarryAhead = 8;

// states[k] = decays[k] states[k - 1] + states[k] over a sequence's segments
// between its first and its last.  grid (quads of a state, sequences on y and z)
__global__ __launch_bounds__(256) void ssm_carry_kernel(SsmArgs a, Segments sg) {
    const int seq = (int)blockIdx.y + (int)blockIdx.z * (int)gridDim.y;
    if (seq >= a.num_seqs) return;
    const long one = (long)a.heads * a.p * a.s, at = ((long)blockIdx.x * 256 + threadIdx.x) * 4;
    const int begin = a.cu_seqlens[seq], all = a.cu_seqlens[seq + 1] - begin;
    const int segs = all > 0 ? (all - 1) / sg.len + 1 : 1;
    if (segs < 3 || at >= one) return;
    const long place = begin / sg.len;
    const float *dec = sg.decays + place * a.heads + at / (a.p * a.s);
    float *p = sg.states + place * one + at;
    f32x4 s = load4(p);
    int k = 1;
    for (; k + kCarryAhead < segs; k += kCarryAhead) {
        f32x4 x[kCarryAhead];
        float d[kCarryAhead];
#pragma unroll
        for (int i = 0; i < kCarryAhead; ++i) {
            x[i] = load4(p + (k + i) * one);
            d[i] = dec[(long)(k + i) * a.heads];
        }
#pragma unroll
        for (int i = 0; i < kCarryAhead; ++i) {
            s = d[i] * s + x[i];
            *reinterpret_cast<f32x4 *>(p + (k + i) * one) = s;
        }
    }
    for (; k < segs - 1; ++k) {
        s = dec[(long)k * a.heads] * s + load4(p + k * one);
        *reinterpret_cast<f32x4 *>(p + k * one) = s;
    }
}

template <int P, int S, typename ST> static hipError_t launch_chunk(const SsmArgs &a, const Segments &sg, hipStream_t s) {
    using C = Chunk<P, S>;
    static_assert(C::LDS <= 163840, "LDS");
    const auto kern = ssm_chunk_kernel<P, S, ST>;
    const hipError_t e = hipFuncSetAttribute((const void *)kern, hipFuncAttributeMaxDynamicSharedMemorySize, C::LDS);
    if (e != hipSuccess) return e;
    kern<<<dim3(ssm_units(a, sg) * ssm_head_workgroups(a)), 256, C::LDS, s>>>(a, sg);
    return hipGetLastError();
}
template <int P, int S> static hipError_t launch_st(const SsmArgs &a, const Segments &sg, hipStream_t s) {
    return a.state_bf16 ? launch_chunk<P, S, bf16>(a, sg, s) : launch_chunk<P, S, float>(a, sg, s);
}
template <int P> static hipError_t launch_s(const SsmArgs &a, const Segments &sg, hipStream_t s) {
    switch (a.s) {
    case 32: return launch_st<P, 32>(a, sg, s);
    case 64: return launch_st<P, 64>(a, sg, s);
    default: return launch_st<P, 128>(a, sg, s);
    }
}
static hipError_t launch_any(const SsmArgs &a, const Segments &sg, hipStream_t s) {
    if (!a.io_bf16) return launch_ssm_chunk_f32(a, sg, s);
    switch (a.p) {
    case 32: return launch_s<32>(a, sg, s);
    case 64: return launch_s<64>(a, sg, s);
    default: return launch_s<128>(a, sg, s);
    }
}

// Tokens of a segment: as many as leave the chip's 512 resident workgroups
// about two segments each, but at least 64 where the sequences by themselves
// are fewer than 64 workgroups, 128 below 128 and else 256 (the launches after
// the first cost more than a shorter chain then saves).  Measured (us) at
// least, S = 128:
//     workgroups                                   64     128     256     512
//      4  1 x 600, 8 heads x 64 (bf16 / fp32)  29 / 60  40 / 98  58 / 171  66 / 207
//      8  1 x 4096, 8 x 128 (bf16)                 54      50      62      95
//     16  8 x 1000, 4 x 64 (bf16)                  40      46      63     102
//     28  7 x 1 .. 300, 8 x 64, S = 64 (fp32)      40      60      56      55
//     64  4 x 512, 32 x 64 (bf16 / fp32)     48 / 101 47 / 107 62 / 179 54 / 171
//     80  20 x 400, 8 x 64 (bf16 / fp32)     50 / 109 48 / 109 58 / 160 50 / 151
//    100  100 x 130, 1 x 128 (bf16 / fp32)    36 / 62  35 / 74  28 / 66  28 / 66
//    120  60 x 500, 4 x 64 (bf16)                  80      60      65      57
//    128  8 x 1000, 32 x 64 (bf16 / fp32)    99 / 304 99 / 304 84 / 277 106 / 339
//    320  20 x 130, 32 x 64 (bf16 / fp32)    68 / 168 52 / 161 42 / 142 43 / 142
static Segments segments_of(int num_seqs, int total_tokens, int head_workgroups) {
    Segments sg{};
    const long len = ((long)total_tokens * head_workgroups / 1024 + 63) / 64 * 64;
    const long alone = (long)num_seqs * head_workgroups, least = alone < 64 ? 64 : alone < 128 ? 128 : 256;
    sg.len = (int)std::min(std::max(len, least), (long)INT32_MAX - 63);
    const bool single = sg.len >= total_tokens;   // every sequence is one segment
    if (single) sg.len = total_tokens > 0 ? total_tokens : 1;
    sg.after = single ? 0 : total_tokens / sg.len;
    return sg;
}
static int head_workgroups(int heads, int groups, int p) {
    const int hw = 128 / p, rep = heads / groups;
    return groups * ((rep + hw - 1) / hw);
}
int ssm_head_workgroups(const SsmArgs &a) { return head_workgroups(a.heads, a.groups, a.p); }
long ssm_prefill_grid(int num_seqs, int total_tokens, int heads, int groups, int p) {
    const int w = head_workgroups(heads, groups, p);
    return ((long)num_seqs + segments_of(num_seqs, total_tokens, w).after) * w;
}

size_t ssm_prefill_workspace_bytes(int num_seqs, int total_tokens, int heads, int groups, int p, int s) {
    if (num_seqs <= 0) return 0;
    const Segments sg = segments_of(num_seqs, total_tokens, head_workgroups(heads, groups, p));
    if (sg.after == 0) return 0;
    return (size_t)sg.after * heads * ((size_t)p * s + 1) * sizeof(float);
}

hipError_t launch_ssm_prefill(const SsmArgs &a, void *workspace, hipStream_t stream) {
    Segments sg = segments_of(a.num_seqs, a.total_tokens, ssm_head_workgroups(a));
    if (sg.after == 0) return launch_any(a, sg, stream);
    const size_t one = (size_t)a.heads * a.p * a.s;
    sg.states = static_cast<float *>(workspace);
    sg.decays = sg.states + sg.after * one;
    hipError_t e = launch_any(a, sg, stream);
    if (e != hipSuccess) return e;
    if (2L * sg.len < a.total_tokens) {   // a sequence of three segments may be there
        ssm_carry_kernel<<<dim3((unsigned)((one / 4 + 255) / 256), decode_grid_y(a.num_seqs), decode_grid_z(a.num_seqs)), 256, 0,
                           stream>>>(a, sg);
        if ((e = hipGetLastError()) != hipSuccess) return e;
    }
    sg.later = true;
    return launch_any(a, sg, stream);
}

}  // namespace kda
