// Selective state-space scan, token by token, against a state pool:
//     S = exp(-exp(A_log) dt) S + dt x B^T;   y = S C + D x;   y *= silu(z)
// one token a request (ssm_token_kernel), or a run of tokens with the state in
// registers (ssm_run_kernel), every state optionally kept in a step cache.
//
// As in the delta rule's decode, a workgroup streams BV stored rows (one row
// per channel p of the head, the S states contiguous) of state[slot, h]; rows
// are independent given B, C and the step.  Bound by the state's bytes, read
// once and written once with 16-byte nontemporal accesses.
//
// Measured: one token of 4096 requests x 32 heads x (128 x 128) 3.00 ms
// (17.3 GB, 5.8 TB/s); of one request 4.3 us, a launch and a row's latency; four
// tokens of 1024 requests x 32 heads x (64 x 128), every state cached, 0.93 ms
// (5.4 GB, 5.8 TB/s, four fifths of it writes).
#include "kda_device.h"
#include "kda_internal.h"
#include "kda_rows.h"
#include "kda_ssm.h"

namespace kda {

// B and C of one (token, group) for states c0 .. c0+VEC-1, and the steps and
// decays of (token, heads h .. h+HD-1).
template <int VEC, typename IO, int HD>
__device__ __forceinline__ void ssm_inputs(const SsmArgs &a, long t, int h, int g, int c0, const float (&A)[HD],
                                           const float (&bias)[HD], float (&Bv)[VEC], float (&Cv)[VEC], float (&step)[HD],
                                           float (&dec)[HD]) {
    const IO *bp = reinterpret_cast<const IO *>(a.B) + t * a.b_stride + (long)g * a.s + c0;
    const IO *cp = reinterpret_cast<const IO *>(a.C) + t * a.c_stride + (long)g * a.s + c0;
#pragma unroll
    for (int i = 0; i < VEC; i += 4) {
        const f32x4 x = load4(bp + i), y = load4(cp + i);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            Bv[i + e] = x[e];
            Cv[i + e] = y[e];
        }
    }
#pragma unroll
    for (int k = 0; k < HD; ++k) {
        step[k] = softplus_f(io_traits<IO>::load(reinterpret_cast<const IO *>(a.dt), t * a.dt_stride + h + k) + bias[k]);
        dec[k] = exp_f(A[k] * step[k]);
    }
}

// A head's constants: the rate (finite, as a step may be 0), the bias of its step
// and D.
template <int HD>
__device__ __forceinline__ void ssm_heads(const SsmArgs &a, int h, float (&A)[HD], float (&bias)[HD], float (&Dh)[HD]) {
#pragma unroll
    for (int k = 0; k < HD; ++k) {
        A[k] = -fminf(expf(a.A_log[h + k]), 3.4e38f);
        bias[k] = a.dt_bias ? a.dt_bias[h + k] : 0.f;
        Dh[k] = a.D ? a.D[h + k] : 0.f;
    }
}

// One token applied to this thread's rows; xrow(p, row) gives x of the
// thread's row of pass p.  Lane cg of a row group writes the output of the
// group's row of pass cg, so the epilogue runs once a lane, not once a row.
// The tile's rows are those of HD heads, one after the other.
template <int DS, int BV, typename IO, typename ST, int HD, typename XF>
__device__ __forceinline__ void ssm_update(XF xrow, const IO *xp, const IO *zp, IO *yp, const float (&Dh)[HD], int r0, int cg,
                                           float (&s)[RowTile<DS, BV, ST>::NP][RowTile<DS, BV, ST>::VEC],
                                           const float (&Bv)[RowTile<DS, BV, ST>::VEC],
                                           const float (&Cv)[RowTile<DS, BV, ST>::VEC], const float (&step)[HD],
                                           const float (&dec)[HD]) {
    using R = RowTile<DS, BV, ST>;
    static_assert(R::NP <= R::LPR, "a lane for every pass");
    static_assert(R::NP % HD == 0, "a pass's rows are one head's");
    const int own = r0 + cg * R::RPP;
    const bool writes = cg < R::NP && own < BV;
    float own_x = 0.f, own_z = 0.f, y = 0.f;
    if (writes) {
        own_x = io_traits<IO>::load(xp, own);
        if (zp) own_z = io_traits<IO>::load(zp, own);
    }
#pragma unroll
    for (int p = 0; p < R::NP; ++p) {
        const int k = p * HD / R::NP;
        const float u = row_in<DS, BV, ST>(r0, p) ? step[k] * xrow(p, r0 + p * R::RPP) : 0.f;
        float acc = 0.f;
#pragma unroll
        for (int i = 0; i < R::VEC; ++i) {
            s[p][i] = s[p][i] * dec[k] + u * Bv[i];
            acc += s[p][i] * Cv[i];
        }
        acc = group_sum<R::LPR>(acc);
        y = cg == p ? acc : y;
    }
    if (writes) {
        y += (cg * HD < R::NP ? Dh[0] : Dh[HD - 1]) * own_x;
        if (zp) y *= own_z * sigmoid_f(own_z);
        io_traits<IO>::store(yp, own, y);
    }
}

template <int DS, int BV, typename IO, typename ST, int HD> __global__ __launch_bounds__(256) void ssm_token_kernel(SsmArgs a) {
    using R = RowTile<DS, BV, ST>;
    const int tid = threadIdx.x, cg = tid % R::LPR, r0 = tid / R::LPR;
    const int nt = HD > 1 ? 1 : a.p / BV;   // row tiles per head
    const int b = (int)blockIdx.y + (int)blockIdx.z * (int)gridDim.y;
    if (b >= a.num_seqs) return;
    const int h = (int)blockIdx.x / nt * HD, j0 = ((int)blockIdx.x % nt) * BV;
    int slot = a.indices[b];
    if (slot < 0) slot = a.num_slots - 1;
    ST *st = reinterpret_cast<ST *>(a.state_out) + (((long)slot * a.heads + h) * a.p + j0) * (long)DS;
    unsigned ro[R::NP];
    row_offs<DS, BV, ST, true>(r0, cg, ro);
    float s[R::NP][R::VEC];
    load_rows<DS, BV, ST, true>(st, ro, r0, s);

    const long hp = (long)h * a.p + j0;
    const IO *xp = reinterpret_cast<const IO *>(a.x) + b * a.x_stride + hp;
    const IO *zp = a.z ? reinterpret_cast<const IO *>(a.z) + b * a.z_stride + hp : nullptr;
    float x[R::NP];   // loaded ahead of the rows' arithmetic: 3.07 -> 3.00 ms for 4096 requests x 32 heads x (128 x 128)
#pragma unroll
    for (int p = 0; p < R::NP; ++p) x[p] = row_in<DS, BV, ST>(r0, p) ? io_traits<IO>::load(xp, r0 + p * R::RPP) : 0.f;
    float Bv[R::VEC], Cv[R::VEC], A[HD], bias[HD], Dh[HD], step[HD], dec[HD];
    ssm_heads(a, h, A, bias, Dh);
    ssm_inputs<R::VEC, IO>(a, b, h, h / (a.heads / a.groups), cg * R::VEC, A, bias, Bv, Cv, step, dec);
    ssm_update<DS, BV, IO, ST>([&](int p, int) { return x[p]; }, xp, zp, reinterpret_cast<IO *>(a.y) + (long)b * a.heads * a.p + hp,
                               Dh, r0, cg, s, Bv, Cv, step, dec);
    store_rows<DS, BV, ST, true>(st, ro, r0, s);
}

// Request n runs tokens [cu[n], cu[n+1]) from its pool row.  Step j's state
// goes to cache[n * pitch + j] for j < cache_steps, the last one to the pool
// where state_out is set.
template <int DS, int BV, typename IO, typename ST, int HD> __global__ __launch_bounds__(256) void ssm_run_kernel(SsmArgs a) {
    using R = RowTile<DS, BV, ST>;
    const int tid = threadIdx.x, cg = tid % R::LPR, r0 = tid / R::LPR;
    const int nt = HD > 1 ? 1 : a.p / BV;
    const int b = (int)blockIdx.y + (int)blockIdx.z * (int)gridDim.y;
    if (b >= a.num_seqs) return;
    const int h = (int)blockIdx.x / nt * HD, j0 = ((int)blockIdx.x % nt) * BV;
    const int t0 = a.cu_seqlens[b], t1 = a.cu_seqlens[b + 1];
    if (t1 <= t0) return;
    long slot = a.indices[b];
    if (slot < 0) slot = a.num_slots - 1;
    const long at = ((slot * a.heads + h) * a.p + j0) * (long)DS;
    unsigned ro[R::NP];
    row_offs<DS, BV, ST>(r0, cg, ro);
    float s[R::NP][R::VEC];
    load_rows<DS, BV, ST, true>(reinterpret_cast<const ST *>(a.state_in) + at, ro, r0, s);

    float A[HD], bias[HD], Dh[HD];
    ssm_heads(a, h, A, bias, Dh);
    const int g = h / (a.heads / a.groups);
    const long hp = (long)h * a.p + j0, step_elems = (long)a.heads * a.p * DS;
    float Bv[R::VEC], Cv[R::VEC], step[HD], dec[HD];
    ssm_inputs<R::VEC, IO>(a, t0, h, g, cg * R::VEC, A, bias, Bv, Cv, step, dec);
    for (int t = t0; t < t1; ++t) {
        // the next token's inputs first (the last token reloads itself); its x
        // too measured slower (1.03 -> 1.08 ms for 1024 x 4 tokens x 32 heads x (64 x 128))
        float Bn[R::VEC], Cn[R::VEC], step_n[HD], dec_n[HD];
        ssm_inputs<R::VEC, IO>(a, min(t + 1, t1 - 1), h, g, cg * R::VEC, A, bias, Bn, Cn, step_n, dec_n);
        const IO *xp = reinterpret_cast<const IO *>(a.x) + t * a.x_stride + hp;
        ssm_update<DS, BV, IO, ST>([&](int, int row) { return io_traits<IO>::load(xp, row); }, xp,
                                   a.z ? reinterpret_cast<const IO *>(a.z) + t * a.z_stride + hp : nullptr,
                                   reinterpret_cast<IO *>(a.y) + (long)t * a.heads * a.p + hp, Dh, r0, cg, s, Bv, Cv, step, dec);
        const int j = t - t0;
        if (a.cache && j < a.cache_steps) {
            ST *cb = reinterpret_cast<ST *>(a.cache) + ((long)b * a.cache_pitch + j) * step_elems + hp * DS;
            const __amdgpu_buffer_rsrc_t cr =
                __builtin_amdgcn_make_buffer_rsrc(cb, 0, BV * DS * (int)sizeof(ST), kBufferWord3);
            store_rows_buf<DS, BV, ST>(cr, ro[0] * (unsigned)sizeof(ST), r0, s);
        }
#pragma unroll
        for (int i = 0; i < R::VEC; ++i) {
            Bv[i] = Bn[i];
            Cv[i] = Cn[i];
        }
#pragma unroll
        for (int k = 0; k < HD; ++k) {
            step[k] = step_n[k];
            dec[k] = dec_n[k];
        }
    }
    if (a.state_out) store_rows<DS, BV, ST, true>(reinterpret_cast<ST *>(a.state_out) + at, ro, r0, s);
}

template <int DS, int BV, typename IO, typename ST> static hipError_t launch_t(const SsmArgs &a, bool run, hipStream_t stream) {
    // Whole heads of 64 rows, two of a group in one workgroup, where a head's
    // state is 32 KB and tokens are run, or 4 KB.  Measured, one head against
    // two a workgroup, 2048 requests of one token (and 1024 of four, every state
    // cached) x 32 heads: rows of 512 bytes 764 / 776 (1077 / 926) us, of 256
    // (fp32) 343 / 394 (499 / 539) and (bf16) 339 / 393 (455 / 495), of 128 168 /
    // 171 (234 / 256), of 64 107 / 86 (190 / 155).
    constexpr int row = DS * (int)sizeof(ST);
    const dim3 grid(a.heads * (a.p / BV), decode_grid_y(a.num_seqs), decode_grid_z(a.num_seqs));
    if constexpr (BV == 64 && (row == 512 || row == 64)) {
        if (a.heads / a.groups % 2 == 0 && (run || row == 64)) {
            const dim3 half(grid.x / 2, grid.y, grid.z);
            if (run) ssm_run_kernel<DS, 128, IO, ST, 2><<<half, 256, 0, stream>>>(a);
            else if constexpr (row == 64) ssm_token_kernel<DS, 128, IO, ST, 2><<<half, 256, 0, stream>>>(a);
            return hipGetLastError();
        }
    }
    if (run) ssm_run_kernel<DS, BV, IO, ST, 1><<<grid, 256, 0, stream>>>(a);
    else ssm_token_kernel<DS, BV, IO, ST, 1><<<grid, 256, 0, stream>>>(a);
    return hipGetLastError();
}
template <int DS, int BV> static hipError_t launch_d(const SsmArgs &a, bool run, hipStream_t s) {
    if (a.io_bf16) return a.state_bf16 ? launch_t<DS, BV, bf16, bf16>(a, run, s) : launch_t<DS, BV, bf16, float>(a, run, s);
    return a.state_bf16 ? launch_t<DS, BV, float, bf16>(a, run, s) : launch_t<DS, BV, float, float>(a, run, s);
}
template <int DS> static hipError_t launch_b(const SsmArgs &a, bool run, hipStream_t s) {
    switch (decode_tile(a.p, a.num_seqs, a.heads, run)) {
    case 32: return launch_d<DS, 32>(a, run, s);
    case 64: return launch_d<DS, 64>(a, run, s);
    default: return launch_d<DS, 128>(a, run, s);
    }
}
static hipError_t launch_s(const SsmArgs &a, bool run, hipStream_t s) {
    switch (a.s) {
    case 32: return launch_b<32>(a, run, s);
    case 64: return launch_b<64>(a, run, s);
    default: return launch_b<128>(a, run, s);
    }
}

hipError_t launch_ssm_decode(const SsmArgs &a, hipStream_t s) { return launch_s(a, false, s); }
hipError_t launch_ssm_multi(const SsmArgs &a, hipStream_t s) { return launch_s(a, true, s); }

}  // namespace kda
