// Internal launch interface between the C ABI (kda_api.hip) and the kernels.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace kda {

struct DecodeArgs {
    const void *q, *k, *v;
    const float *g, *beta;             // activated gate and beta (fp32), or
    const void *gx, *bx;               // raw gate and beta inputs (io dtype) with
    const float *A_log, *dt_bias;      // per-(head, channel) activation parameters
    void *state;
    const int32_t *indices;
    void *o;
    int batch, hk, hv, dk, dv, num_slots;
    float scale;
    bool io_bf16, state_bf16, scalar_gate, raw_gate;
    // token row strides (elements) of q, k (same stride) and v: hk * dk and hv * dv
    // for separate tensors, 2 hk dk + hv dv for one packed [q | k | v] row per token
    long qk_stride, v_stride;
    // multi-token decode only: request n owns tokens [cu_seqlens[n], cu_seqlens[n+1]);
    // the state after its step j goes to cache[n * cache_pitch + j] when j < cache_pitch
    const int32_t *cu_seqlens;
    void *cache;
    int cache_pitch;
    bool update_pool;
};

hipError_t launch_decode(const DecodeArgs &a, hipStream_t stream);
hipError_t launch_decode_multi(const DecodeArgs &a, hipStream_t stream);
int decode_tile(int dv, long batch, int hv, bool multi);
int decode_grid_y(int batch);   // requests per z slab of the decode grid
int decode_grid_z(int batch);   // z slabs

// Chunked prefill.  Chunk size and the chunk-slot bound are fixed here.
constexpr int kChunk = 64;

struct PrefillArgs {
    const void *q, *k, *v;
    const float *g, *beta;             // activated gate and beta (fp32), or
    const void *gx, *bx;               // raw gate and beta inputs (io dtype) with
    const float *A_log, *dt_bias;      // per-(head, channel) activation parameters
    const int32_t *cu_seqlens;
    const void *state_in;     // dense h0, pool, or NULL
    void *state_out;          // dense ht, pool, or NULL
    const int32_t *indices;   // pool slots or NULL
    void *o;
    int num_seqs, total_tokens, hk, hv, dk, dv, num_slots;
    float scale;
    bool io_bf16, state_bf16, scalar_gate, raw_gate;
};


size_t prefill_workspace_bytes(int num_seqs, int total_tokens, int hv, int dk, int dv);
hipError_t launch_prefill(PrefillArgs &a, void *workspace, hipStream_t stream);

// Short causal convolution.
struct ConvArgs {
    const void *x, *weight, *bias;
    const int32_t *cu_seqlens;
    const void *state_in;     // dense states, pool, or NULL (zeros)
    void *state_out;          // dense states, pool, or NULL (not written)
    const int32_t *indices;   // pool slots or NULL
    const int32_t *steps;     // commit only
    void *y;
    int num_seqs, total_tokens, channels, width, num_slots;
    bool io_bf16, silu;
    long x_stride;
};
hipError_t launch_conv_prefill(const ConvArgs &a, hipStream_t stream);
hipError_t launch_conv_decode(const ConvArgs &a, hipStream_t stream);
hipError_t launch_conv_commit(const ConvArgs &a, hipStream_t stream);
long conv_prefill_tiles(int num_seqs, int total_tokens);   // workgroup rows of the prefill grid

// Selective state-space scan.
struct SsmArgs {
    const void *x, *dt, *B, *C, *z;
    const float *A_log, *D, *dt_bias;
    const int32_t *cu_seqlens;   // NULL: one token a request
    const void *state_in;        // dense states, pool, or NULL (zeros)
    void *state_out;             // dense states, pool, or NULL (not written)
    const int32_t *indices;
    void *cache;                 // step cache or NULL
    void *y;
    int num_seqs, total_tokens, heads, groups, p, s, num_slots, cache_steps, cache_pitch;
    bool io_bf16, state_bf16;
    long x_stride, dt_stride, b_stride, c_stride, z_stride;
};
hipError_t launch_ssm_decode(const SsmArgs &a, hipStream_t stream);
hipError_t launch_ssm_multi(const SsmArgs &a, hipStream_t stream);
hipError_t launch_ssm_prefill(const SsmArgs &a, void *workspace, hipStream_t stream);
long ssm_prefill_grid(int num_seqs, int total_tokens, int heads, int groups, int p);   // workgroups of a launch
size_t ssm_prefill_workspace_bytes(int num_seqs, int total_tokens, int heads, int groups, int p, int s);

// Draft verification and commit.
struct VerifyArgs {
    const int32_t *tokens, *cu_seqlens;
    const void *target, *draft;
    const float *uniform, *uniform_next;
    int32_t *accepted, *next, *emitted;
    double *partial;             // [N] verdicts (8 bytes each), then [N, 2, parts] sums
    int num_seqs, vocab, parts;
    bool bf16;
    long target_stride, draft_stride;
};
int verify_parts(int vocab);
hipError_t launch_verify(const VerifyArgs &a, hipStream_t stream);
hipError_t launch_commit(const int32_t *indices, const int32_t *steps, const void *cache, void *pool, int num_seqs,
                         int num_slots, int cache_steps, int cache_pitch, long row_bytes, hipStream_t stream);

}  // namespace kda
