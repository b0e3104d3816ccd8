// Streaming of stored state rows ([V, K] or [P, N], the inner axis contiguous)
// between a workgroup's registers and memory, shared by the decode kernels.
#pragma once

#include "kda_device.h"

namespace kda {

// Thread layout over one workgroup's BV stored rows: LPR lanes per row, each
// holding VEC consecutive channels (16 bytes of state); NP passes of RPP rows.
template <int DK, int BV, typename ST> struct RowTile {
    static constexpr int VEC = (sizeof(ST) == 4) ? 4 : 8;  // state elements per 16 B
    static constexpr int LPR = DK / VEC;                    // lanes per stored row
    static constexpr int RPP = 256 / LPR;                   // rows per pass
    static constexpr int NP = (BV + RPP - 1) / RPP;         // passes
    static_assert(DK % VEC == 0 && LPR <= 64, "tile");
};

// Element offsets of this thread's rows within a block of BV stored rows.
// With OPAQUE they are formed once and hidden from the compiler, which
// otherwise re-forms the row addresses between the row stores at the end of
// the one-token decode; the stores then go out back to back (measured 3.7%
// faster for the B = 4096 decode).
template <int DK, int BV, typename ST, bool OPAQUE = false>
__device__ __forceinline__ void row_offs(int r0, int cg, unsigned (&ro)[RowTile<DK, BV, ST>::NP]) {
    using R = RowTile<DK, BV, ST>;
#pragma unroll
    for (int p = 0; p < R::NP; ++p) {
        ro[p] = (unsigned)((r0 + p * R::RPP) * DK + cg * R::VEC);
        if constexpr (OPAQUE) asm volatile("" : "+v"(ro[p]));
    }
}

// Whether pass p holds a row of the block (always, when the passes tile it).
template <int DK, int BV, typename ST> __device__ __forceinline__ bool row_in(int r0, int p) {
    using R = RowTile<DK, BV, ST>;
    return R::NP * R::RPP == BV || r0 + p * R::RPP < BV;
}

// Load this thread's part of the rows at st (offsets ro) into s.
template <int DK, int BV, typename ST, bool NT>
__device__ __forceinline__ void load_rows(const ST *st, const unsigned (&ro)[RowTile<DK, BV, ST>::NP], int r0,
                                          float (&s)[RowTile<DK, BV, ST>::NP][RowTile<DK, BV, ST>::VEC]) {
    using R = RowTile<DK, BV, ST>;
#pragma unroll
    for (int p = 0; p < R::NP; ++p) {
        if (row_in<DK, BV, ST>(r0, p)) {
            const ST *src = st + ro[p];
            if constexpr (R::VEC == 4) {
                f32x4 x = NT ? __builtin_nontemporal_load(reinterpret_cast<const f32x4 *>(src)) : load4(src);
#pragma unroll
                for (int i = 0; i < 4; ++i) s[p][i] = x[i];
            } else {
                u32x4 w = NT ? __builtin_nontemporal_load(reinterpret_cast<const u32x4 *>(src))
                             : *reinterpret_cast<const u32x4 *>(src);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    s[p][2 * i] = __uint_as_float(w[i] << 16);
                    s[p][2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
                }
            }
        }
    }
}

// Store this thread's part of the rows to st (offsets ro; bf16 storage rounds
// to nearest even).
template <int DK, int BV, typename ST, bool NT>
__device__ __forceinline__ void store_rows(ST *st, const unsigned (&ro)[RowTile<DK, BV, ST>::NP], int r0,
                                           const float (&s)[RowTile<DK, BV, ST>::NP][RowTile<DK, BV, ST>::VEC]) {
    using R = RowTile<DK, BV, ST>;
#pragma unroll
    for (int p = 0; p < R::NP; ++p) {
        if (row_in<DK, BV, ST>(r0, p)) {
            ST *dst = st + ro[p];
            if constexpr (R::VEC == 4) {
                f32x4 x;
#pragma unroll
                for (int i = 0; i < 4; ++i) x[i] = s[p][i];
                if constexpr (NT) __builtin_nontemporal_store(x, reinterpret_cast<f32x4 *>(dst));
                else *reinterpret_cast<f32x4 *>(dst) = x;
            } else {
                u32x4 w;
#pragma unroll
                for (int i = 0; i < 4; ++i) w[i] = pack_bf16x2(s[p][2 * i], s[p][2 * i + 1]);
                if constexpr (NT) __builtin_nontemporal_store(w, reinterpret_cast<u32x4 *>(dst));
                else *reinterpret_cast<u32x4 *>(dst) = w;
            }
        }
    }
}

// Cache policy of the state stores that stream out of the verify decode: the
// nontemporal and device-scope bits (nt, sc1).  Its cached steps measured on
// MI355X (1024 requests x 4 tokens): nt alone 1.885 ms, nt with sc1
// 1.842 ms, sc0 with sc1 and no nt 2.10 ms.
constexpr int kStreamStore = 2 | 16;

// Store this thread's part of the rows through a buffer resource covering the
// row block: the lane's offset is one register and each pass adds a scalar
// offset, so the stores need no address arithmetic between them and go out
// back to back; the range check bounds them to the block.
//
// A store with its offset in a scalar register reads its data late, but the
// compiler takes it to be read at once: a vector instruction right behind one
// that wrote a register of the data has changed what the last quarter of the
// lanes stored.  So all data are formed first, in registers of their own, no
// instruction is moved between the stores, and wait states follow the last.
// (Wait states after each store, or a resource a pass in place of the offsets,
// cost the verify decode of 1024 x 4 tokens 4%, 1.92 against 1.84 ms.)
template <int DK, int BV, typename ST>
__device__ __forceinline__ void store_rows_buf(const __amdgpu_buffer_rsrc_t rsrc, unsigned voff, int r0,
                                               const float (&s)[RowTile<DK, BV, ST>::NP][RowTile<DK, BV, ST>::VEC]) {
    using R = RowTile<DK, BV, ST>;
    u32x4 w[R::NP];
#pragma unroll
    for (int p = 0; p < R::NP; ++p) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (R::VEC == 4) w[p][i] = __float_as_uint(s[p][i]);
            else w[p][i] = pack_bf16x2(s[p][2 * i], s[p][2 * i + 1]);
        }
    }
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int p = 0; p < R::NP; ++p)
        if (row_in<DK, BV, ST>(r0, p))
            __builtin_amdgcn_raw_buffer_store_b128(w[p], rsrc, voff, p * R::RPP * DK * (int)sizeof(ST), kStreamStore);
    asm volatile("s_nop 7" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
}

}  // namespace kda
