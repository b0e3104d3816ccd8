// C ABI of the convolution, state-space scan, draft verification and commit:
// host-side validation and launch.  The contract lives in include/kda.h.
#include <hip/hip_runtime.h>

#include "kda_check.h"
#include "kda_internal.h"

namespace {

using namespace kda;

struct Range { const void *p; size_t n; };

// Bytes from the first to the last element of `rows` token rows of `width`
// elements, `stride` elements apart.
size_t rows_bytes(long rows, long stride, long width, size_t isz) {
    return rows <= 0 ? 0 : ((size_t)(rows - 1) * (size_t)stride + (size_t)width) * isz;
}

template <int N> bool all_aligned(const void *const (&ptrs)[N]) {
    for (const void *p : ptrs)
        if (p && !aligned(p)) return false;
    return true;
}

template <int N> bool hits(const Range &out, const Range (&ins)[N]) {
    for (const Range &r : ins)
        if (overlap(out.p, out.n, r.p, r.n)) return true;
    return false;
}

// Grid (x, rows over y and z) within the current device's limits?
kda_status grid_ok(long x, long rows) {
    int dev = 0, mx = 0, my = 0, mz = 0;
    if (hipGetDevice(&dev) != hipSuccess || hipDeviceGetAttribute(&mx, hipDeviceAttributeMaxGridDimX, dev) != hipSuccess ||
        hipDeviceGetAttribute(&my, hipDeviceAttributeMaxGridDimY, dev) != hipSuccess ||
        hipDeviceGetAttribute(&mz, hipDeviceAttributeMaxGridDimZ, dev) != hipSuccess)
        return KDA_ERR_HIP;
    if (x > mx || rows > INT32_MAX || decode_grid_y((int)rows) > my || decode_grid_z((int)rows) > mz) return KDA_ERR_UNSUPPORTED;
    return KDA_OK;
}

// ---- convolution -----------------------------------------------------------

kda_status check_conv(const kda_conv_desc *d, bool pool) {
    if (!d) return KDA_ERR_NULL;
    if (d->num_seqs < 0 || d->total_tokens < 0 || d->channels <= 0 || d->x_stride < d->channels || (pool && d->num_slots <= 0))
        return KDA_ERR_SHAPE;
    if (d->width < 2 || d->width > 4 || !dtype_ok(d->io_dtype) || d->channels > (1 << 28)) return KDA_ERR_UNSUPPORTED;
    return KDA_OK;
}

ConvArgs conv_args(const kda_conv_desc *d) {
    ConvArgs a{};
    a.num_seqs = d->num_seqs;
    a.total_tokens = d->total_tokens;
    a.channels = d->channels;
    a.width = d->width;
    a.num_slots = d->num_slots;
    a.io_bf16 = d->io_dtype == KDA_BF16;
    a.silu = d->silu != 0;
    a.x_stride = d->x_stride;
    return a;
}

size_t conv_states(const kda_conv_desc *d, long rows) {
    return (size_t)rows * (d->width - 1) * d->channels * io_size(d->io_dtype);
}

// ---- scan ------------------------------------------------------------------

kda_status check_ssm(const kda_ssm_desc *d, bool pool) {
    if (!d) return KDA_ERR_NULL;
    if (d->num_seqs < 0 || d->total_tokens < 0 || d->heads <= 0 || d->groups <= 0 || d->head_dim <= 0 || d->state_dim <= 0 ||
        d->heads % d->groups != 0 || (pool && d->num_slots <= 0))
        return KDA_ERR_SHAPE;
    if (!dim_ok(d->head_dim) || !dim_ok(d->state_dim) || !dtype_ok(d->io_dtype) || !dtype_ok(d->state_dtype))
        return KDA_ERR_UNSUPPORTED;
    const long hp = (long)d->heads * d->head_dim, gs = (long)d->groups * d->state_dim;
    if (d->x_stride < hp || d->dt_stride < d->heads || d->b_stride < gs || d->c_stride < gs || d->z_stride < 0) return KDA_ERR_SHAPE;
    // 64 rows stay within a buffer resource's 31 bits
    const int64_t far = 1 << 22;
    if (d->x_stride > far || d->b_stride > far || d->c_stride > far || d->z_stride > far) return KDA_ERR_UNSUPPORTED;
    return KDA_OK;
}

struct SsmIn {
    const void *x, *dt, *B, *C, *z;
    const float *A_log, *D, *dt_bias;
};

// The checks the three scan calls share, for T tokens; fills `a`.  more: what
// else is read or written; the states that are written and the cache or the
// workspace (`extra`) overlap no input, y overlaps nothing.
kda_status ssm_common(const kda_ssm_desc *d, const SsmIn &in, long T, const void *y, const Range (&more)[5], const Range &states,
                      const Range &extra, SsmArgs &a) {
    if (T > 0 && (!in.x || !in.dt || !in.A_log || !in.B || !in.C || !y)) return KDA_ERR_NULL;
    const long hp = (long)d->heads * d->head_dim, gs = (long)d->groups * d->state_dim;
    if (in.z && d->z_stride < hp) return KDA_ERR_SHAPE;
    const void *const ptrs[] = {in.x, in.dt, in.A_log, in.B, in.C, in.D, in.z, in.dt_bias, y};
    if (!all_aligned(ptrs)) return KDA_ERR_ALIGN;
    for (const Range &r : more)
        if (r.p && !aligned(r.p)) return KDA_ERR_ALIGN;
    const size_t isz = io_size(d->io_dtype);
    const long vec = (long)(16 / isz);
    if (T > 1 && (d->x_stride % vec || d->b_stride % vec || d->c_stride % vec)) return KDA_ERR_ALIGN;
    // z comes from a projection beside dt, whose heads may be any number; its loads want whole words
    if (T > 1 && in.z && d->z_stride * (long)isz % 4) return KDA_ERR_ALIGN;
    const Range out{y, (size_t)T * hp * isz};
    const Range ins[] = {{in.x, rows_bytes(T, d->x_stride, hp, isz)}, {in.dt, rows_bytes(T, d->dt_stride, d->heads, isz)},
                         {in.B, rows_bytes(T, d->b_stride, gs, isz)}, {in.C, rows_bytes(T, d->c_stride, gs, isz)},
                         {in.z, in.z ? rows_bytes(T, d->z_stride, hp, isz) : 0}, {in.A_log, (size_t)d->heads * 4},
                         {in.D, (size_t)d->heads * 4}, {in.dt_bias, (size_t)d->heads * 4}};
    if (hits(out, ins) || hits(out, more) || hits(states, ins) || hits(extra, ins)) return KDA_ERR_ALIAS;
    a = SsmArgs{};
    a.x = in.x; a.dt = in.dt; a.B = in.B; a.C = in.C; a.z = in.z;
    a.A_log = in.A_log; a.D = in.D; a.dt_bias = in.dt_bias;
    a.y = const_cast<void *>(y);
    a.num_seqs = d->num_seqs;
    a.total_tokens = (int)T;
    a.heads = d->heads; a.groups = d->groups; a.p = d->head_dim; a.s = d->state_dim;
    a.num_slots = d->num_slots;
    a.io_bf16 = d->io_dtype == KDA_BF16;
    a.state_bf16 = d->state_dtype == KDA_BF16;
    a.x_stride = d->x_stride; a.dt_stride = d->dt_stride; a.b_stride = d->b_stride; a.c_stride = d->c_stride;
    a.z_stride = d->z_stride;
    return KDA_OK;
}

size_t ssm_states(const kda_ssm_desc *d, long rows) {
    return (size_t)rows * d->heads * d->head_dim * d->state_dim * io_size(d->state_dtype);
}

// ---- drafts ----------------------------------------------------------------

kda_status check_verify(const kda_verify_desc *d) {
    if (!d) return KDA_ERR_NULL;
    if (d->num_seqs < 0 || d->total_tokens < 0 || d->vocab <= 0 || d->target_stride < d->vocab) return KDA_ERR_SHAPE;
    if (!dtype_ok(d->prob_dtype) || d->vocab > (1 << 30)) return KDA_ERR_UNSUPPORTED;
    return KDA_OK;
}

}  // namespace

extern "C" {

kda_status kda_conv_prefill(const kda_conv_desc *d, const void *x, const void *weight, const void *bias,
                            const int32_t *cu_seqlens, void *state, const int32_t *state_indices, void *final_state, void *y,
                            void *stream) {
    const bool pool = state_indices != nullptr;
    const kda_status st = check_conv(d, pool);
    if (st != KDA_OK) return st;
    const long T = d->total_tokens, N = d->num_seqs;
    if (!cu_seqlens || !weight || (T > 0 && (!x || !y)) || (pool && !state)) return KDA_ERR_NULL;
    if (pool && final_state && final_state != state) return KDA_ERR_ALIAS;
    const void *const ptrs[] = {x, weight, bias, cu_seqlens, state, state_indices, final_state, y};
    if (!all_aligned(ptrs)) return KDA_ERR_ALIGN;
    const size_t isz = io_size(d->io_dtype), D = d->channels;
    const Range out{y, (size_t)T * D * isz}, last{pool ? nullptr : final_state, conv_states(d, N)};
    const Range ins[] = {{x, rows_bytes(T, d->x_stride, D, isz)}, {weight, D * d->width * isz}, {bias, D * isz},
                         {cu_seqlens, (size_t)(N + 1) * 4}, {state_indices, (size_t)N * 4}};
    const Range before{state, conv_states(d, pool ? d->num_slots : N)};
    const Range written = !pool ? last : d->update_pool ? before : Range{};
    if (hits(out, ins) || overlap(y, out.n, state, before.n) || hits(written, ins) || overlap(last.p, last.n, y, out.n))
        return KDA_ERR_ALIAS;
    if (last.p && last.p != state && overlap(last.p, last.n, state, before.n)) return KDA_ERR_ALIAS;
    if (N == 0 || (T == 0 && (pool || !final_state))) return KDA_OK;
    const kda_status gs = grid_ok((d->channels + 255L) / 256, conv_prefill_tiles(d->num_seqs, d->total_tokens));
    if (gs != KDA_OK) return gs;
    ConvArgs a = conv_args(d);
    a.x = x; a.weight = weight; a.bias = bias; a.cu_seqlens = cu_seqlens;
    a.state_in = state;
    a.state_out = pool ? (d->update_pool ? state : nullptr) : final_state;
    a.indices = state_indices;
    a.y = y;
    return hip_status(launch_conv_prefill(a, static_cast<hipStream_t>(stream)));
}

kda_status kda_conv_decode(const kda_conv_desc *d, const void *x, const void *weight, const void *bias, void *state_pool,
                           const int32_t *state_indices, void *y, void *stream) {
    const kda_status st = check_conv(d, true);
    if (st != KDA_OK) return st;
    const long B = d->num_seqs;
    if (B == 0) return KDA_OK;
    if (!x || !weight || !state_pool || !state_indices || !y) return KDA_ERR_NULL;
    const void *const ptrs[] = {x, weight, bias, state_pool, state_indices, y};
    if (!all_aligned(ptrs)) return KDA_ERR_ALIGN;
    const size_t isz = io_size(d->io_dtype), D = d->channels;
    const Range out{y, (size_t)B * D * isz}, pool{state_pool, conv_states(d, d->num_slots)};
    const Range ins[] = {{x, rows_bytes(B, d->x_stride, D, isz)}, {weight, D * d->width * isz}, {bias, D * isz},
                         {state_indices, (size_t)B * 4}};
    if (hits(out, ins) || hits(pool, ins) || overlap(y, out.n, state_pool, pool.n)) return KDA_ERR_ALIAS;
    const kda_status gs = grid_ok((d->channels + 255L) / 256, B);
    if (gs != KDA_OK) return gs;
    ConvArgs a = conv_args(d);
    a.x = x; a.weight = weight; a.bias = bias;
    a.state_in = state_pool;
    a.state_out = state_pool;
    a.indices = state_indices;
    a.y = y;
    return hip_status(launch_conv_decode(a, static_cast<hipStream_t>(stream)));
}

kda_status kda_conv_commit(const kda_conv_desc *d, const void *x, const int32_t *cu_seqlens, const int32_t *steps,
                           void *state_pool, const int32_t *state_indices, void *stream) {
    const kda_status st = check_conv(d, true);
    if (st != KDA_OK) return st;
    const long T = d->total_tokens, N = d->num_seqs;
    if (N == 0) return KDA_OK;
    if (!cu_seqlens || !steps || !state_pool || !state_indices || (T > 0 && !x)) return KDA_ERR_NULL;
    const void *const ptrs[] = {x, cu_seqlens, steps, state_pool, state_indices};
    if (!all_aligned(ptrs)) return KDA_ERR_ALIGN;
    const Range pool{state_pool, conv_states(d, d->num_slots)};
    const Range ins[] = {{x, rows_bytes(T, d->x_stride, d->channels, io_size(d->io_dtype))}, {cu_seqlens, (size_t)(N + 1) * 4},
                         {steps, (size_t)N * 4}, {state_indices, (size_t)N * 4}};
    if (hits(pool, ins)) return KDA_ERR_ALIAS;
    if (T == 0) return KDA_OK;
    const kda_status gs = grid_ok((d->channels + 255L) / 256, N);
    if (gs != KDA_OK) return gs;
    ConvArgs a = conv_args(d);
    a.x = x; a.cu_seqlens = cu_seqlens; a.steps = steps;
    a.state_out = state_pool;
    a.indices = state_indices;
    return hip_status(launch_conv_commit(a, static_cast<hipStream_t>(stream)));
}

size_t kda_ssm_prefill_workspace_size(const kda_ssm_desc *d) {
    if (check_ssm(d, false) != KDA_OK) return 0;
    return ssm_prefill_workspace_bytes(d->num_seqs, d->total_tokens, d->heads, d->groups, d->head_dim, d->state_dim);
}

kda_status kda_ssm_prefill(const kda_ssm_desc *d, const void *x, const void *dt, const float *A_log, const void *B, const void *C,
                           const float *D, const void *z, const float *dt_bias, const int32_t *cu_seqlens, void *state,
                           const int32_t *state_indices, void *final_state, void *y, void *workspace, size_t workspace_bytes,
                           void *stream) {
    const bool pool = state_indices != nullptr;
    kda_status st = check_ssm(d, pool);
    if (st != KDA_OK) return st;
    const long T = d->total_tokens, N = d->num_seqs;
    if (!cu_seqlens || (pool && !state)) return KDA_ERR_NULL;
    if (pool && final_state && final_state != state) return KDA_ERR_ALIAS;
    const size_t need = ssm_prefill_workspace_bytes(d->num_seqs, d->total_tokens, d->heads, d->groups, d->head_dim, d->state_dim);
    const Range before{state, ssm_states(d, pool ? d->num_slots : N)}, last{pool ? nullptr : final_state, ssm_states(d, N)};
    const Range more[5] = {before, last, {cu_seqlens, (size_t)(N + 1) * 4}, {state_indices, (size_t)N * 4}, {workspace, need}};
    SsmArgs a;
    st = ssm_common(d, SsmIn{x, dt, B, C, z, A_log, D, dt_bias}, T, y, more, pool ? before : last, more[4], a);
    if (st != KDA_OK) return st;
    if (need > 0 && (!workspace || workspace_bytes < need)) return KDA_ERR_WORKSPACE;
    // (the workspace is written while inputs, offsets and first states are still to be read)
    const Range written = pool ? before : last, offsets[] = {more[2], more[3]};
    if (hits(written, offsets) || hits(more[4], offsets) || overlap(written.p, written.n, workspace, need) ||
        overlap(before.p, before.n, workspace, need) || (last.p && last.p != state && overlap(last.p, last.n, state, before.n)))
        return KDA_ERR_ALIAS;
    if (N == 0 || (T == 0 && (pool || !final_state))) return KDA_OK;
    st = grid_ok(ssm_prefill_grid(d->num_seqs, d->total_tokens, d->heads, d->groups, d->head_dim), N);
    if (st != KDA_OK) return st;
    a.cu_seqlens = cu_seqlens;
    a.state_in = state;
    a.state_out = pool ? state : final_state;
    a.indices = state_indices;
    return hip_status(launch_ssm_prefill(a, workspace, static_cast<hipStream_t>(stream)));
}

kda_status kda_ssm_decode(const kda_ssm_desc *d, const void *x, const void *dt, const float *A_log, const void *B, const void *C,
                          const float *D, const void *z, const float *dt_bias, void *state_pool, const int32_t *state_indices,
                          void *y, void *stream) {
    kda_status st = check_ssm(d, true);
    if (st != KDA_OK) return st;
    const long n = d->num_seqs;
    if (n == 0) return KDA_OK;
    if (!state_pool || !state_indices) return KDA_ERR_NULL;
    const Range more[5] = {{state_pool, ssm_states(d, d->num_slots)}, {state_indices, (size_t)n * 4}, {}, {}, {}};
    SsmArgs a;
    st = ssm_common(d, SsmIn{x, dt, B, C, z, A_log, D, dt_bias}, n, y, more, more[0], {}, a);
    if (st != KDA_OK) return st;
    if (overlap(state_pool, more[0].n, state_indices, more[1].n)) return KDA_ERR_ALIAS;
    st = grid_ok((long)d->heads * (d->head_dim / 32), n);
    if (st != KDA_OK) return st;
    a.state_in = state_pool;
    a.state_out = state_pool;
    a.indices = state_indices;
    return hip_status(launch_ssm_decode(a, static_cast<hipStream_t>(stream)));
}

kda_status kda_ssm_decode_multi(const kda_ssm_desc *d, const void *x, const void *dt, const float *A_log, const void *B,
                                const void *C, const float *D, const void *z, const float *dt_bias, const int32_t *cu_seqlens,
                                void *state_pool, const int32_t *state_indices, void *intermediate_states, void *y,
                                void *stream) {
    kda_status st = check_ssm(d, true);
    if (st != KDA_OK) return st;
    if (d->cache_steps < 0 || d->cache_pitch < d->cache_steps) return KDA_ERR_SHAPE;
    const long T = d->total_tokens, N = d->num_seqs;
    if (N == 0) return KDA_OK;
    void *cache = d->cache_steps > 0 ? intermediate_states : nullptr;
    if (!cu_seqlens || !state_pool || !state_indices || (d->cache_steps > 0 && !cache)) return KDA_ERR_NULL;
    const Range kept{cache, cache ? ssm_states(d, (N - 1) * (long)d->cache_pitch + d->cache_steps) : 0};
    const Range more[5] = {{state_pool, ssm_states(d, d->num_slots)}, {state_indices, (size_t)N * 4},
                           {cu_seqlens, (size_t)(N + 1) * 4}, kept, {}};
    SsmArgs a;
    st = ssm_common(d, SsmIn{x, dt, B, C, z, A_log, D, dt_bias}, T, y, more, d->update_pool ? more[0] : Range{}, kept, a);
    if (st != KDA_OK) return st;
    for (int i = 0; i < 3; ++i)
        if (overlap(kept.p, kept.n, more[i].p, more[i].n) || (i > 0 && d->update_pool && overlap(state_pool, more[0].n, more[i].p, more[i].n)))
            return KDA_ERR_ALIAS;
    if (T == 0) return KDA_OK;
    st = grid_ok((long)d->heads * (d->head_dim / 32), N);
    if (st != KDA_OK) return st;
    a.cu_seqlens = cu_seqlens;
    a.state_in = state_pool;
    a.state_out = d->update_pool ? state_pool : nullptr;
    a.indices = state_indices;
    a.cache = cache;
    a.cache_steps = d->cache_steps;
    a.cache_pitch = d->cache_pitch;
    return hip_status(launch_ssm_multi(a, static_cast<hipStream_t>(stream)));
}

size_t kda_verify_drafts_workspace_size(const kda_verify_desc *d) {
    if (check_verify(d) != KDA_OK) return 0;
    return (size_t)d->num_seqs * (1 + 2 * (size_t)verify_parts(d->vocab)) * sizeof(double);
}

kda_status kda_verify_drafts(const kda_verify_desc *d, const int32_t *tokens, const void *target_probs, const void *draft_probs,
                             const int32_t *cu_seqlens, const float *uniform, const float *uniform_next, int32_t *accepted,
                             int32_t *next_tokens, int32_t *emitted, void *workspace, size_t workspace_bytes, void *stream) {
    const kda_status st = check_verify(d);
    if (st != KDA_OK) return st;
    const long T = d->total_tokens, N = d->num_seqs;
    if (draft_probs && d->draft_stride < d->vocab) return KDA_ERR_SHAPE;
    if (N == 0) return KDA_OK;
    if (!cu_seqlens || !uniform_next || !accepted || !next_tokens || (T > 0 && (!tokens || !target_probs || !uniform || !emitted)))
        return KDA_ERR_NULL;
    const void *const ptrs[] = {tokens, target_probs, draft_probs, cu_seqlens, uniform, uniform_next, accepted, next_tokens, emitted,
                                workspace};
    if (!all_aligned(ptrs)) return KDA_ERR_ALIGN;
    const size_t need = kda_verify_drafts_workspace_size(d), psz = io_size(d->prob_dtype);
    if (!workspace || workspace_bytes < need) return KDA_ERR_WORKSPACE;
    const Range outs[] = {{accepted, (size_t)N * 4}, {next_tokens, (size_t)N * 4}, {emitted, (size_t)T * 4}, {workspace, need}};
    const Range ins[] = {{tokens, (size_t)T * 4}, {target_probs, rows_bytes(T, d->target_stride, d->vocab, psz)},
                         {draft_probs, draft_probs ? rows_bytes(T, d->draft_stride, d->vocab, psz) : 0},
                         {cu_seqlens, (size_t)(N + 1) * 4}, {uniform, (size_t)T * 4}, {uniform_next, (size_t)N * 4}};
    for (int i = 0; i < 4; ++i) {
        if (hits(outs[i], ins)) return KDA_ERR_ALIAS;
        for (int j = 0; j < i; ++j)
            if (overlap(outs[i].p, outs[i].n, outs[j].p, outs[j].n)) return KDA_ERR_ALIAS;
    }
    const kda_status gs = grid_ok(1024, N);
    if (gs != KDA_OK) return gs;
    VerifyArgs a{};
    a.tokens = tokens; a.cu_seqlens = cu_seqlens;
    a.target = target_probs; a.draft = draft_probs;
    a.uniform = uniform; a.uniform_next = uniform_next;
    a.accepted = accepted; a.next = next_tokens; a.emitted = emitted;
    a.partial = static_cast<double *>(workspace);
    a.num_seqs = d->num_seqs; a.vocab = d->vocab;
    a.parts = verify_parts(d->vocab);
    a.bf16 = d->prob_dtype == KDA_BF16;
    a.target_stride = d->target_stride; a.draft_stride = d->draft_stride;
    return hip_status(launch_verify(a, static_cast<hipStream_t>(stream)));
}

kda_status kda_commit_states(const kda_commit_desc *d, void *state_pool, const int32_t *state_indices,
                             const void *intermediate_states, const int32_t *steps, void *stream) {
    if (!d) return KDA_ERR_NULL;
    if (d->num_seqs < 0 || d->num_slots <= 0 || d->cache_steps < 0 || d->cache_pitch < d->cache_steps || d->row_bytes <= 0 ||
        d->row_bytes % 16 != 0)
        return KDA_ERR_SHAPE;
    const long N = d->num_seqs;
    if (N == 0 || d->cache_steps == 0) return KDA_OK;
    if (!state_pool || !state_indices || !intermediate_states || !steps) return KDA_ERR_NULL;
    const void *const ptrs[] = {state_pool, state_indices, intermediate_states, steps};
    if (!all_aligned(ptrs)) return KDA_ERR_ALIGN;
    const Range pool{state_pool, (size_t)d->num_slots * d->row_bytes};
    const Range ins[] = {{state_indices, (size_t)N * 4}, {steps, (size_t)N * 4},
                         {intermediate_states, (size_t)((N - 1) * (long)d->cache_pitch + d->cache_steps) * d->row_bytes}};
    if (hits(pool, ins)) return KDA_ERR_ALIAS;
    const kda_status gs = grid_ok((d->row_bytes + 4095) / 4096, N);
    if (gs != KDA_OK) return gs;
    return hip_status(launch_commit(state_indices, steps, intermediate_states, state_pool, d->num_seqs, d->num_slots, d->cache_steps,
                                    d->cache_pitch, d->row_bytes, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
