// C ABI of the paged cache, the attention over it and the choice of the next
// token: host-side validation and launch.  The contract lives in include/kda.h.
#include <hip/hip_runtime.h>

#include "kda_check.h"
#include "kda_internal.h"

namespace {

using namespace kda;

// What a call reads or writes: where, how many bytes, and what its address is a
// multiple of.
struct Span { const void *p; size_t n; unsigned align; };

size_t rows_bytes(long rows, long stride, long width, size_t isz) {
    return rows <= 0 ? 0 : ((size_t)(rows - 1) * (size_t)stride + (size_t)width) * isz;
}

// Alignment of all, and that no output overlaps an input or another output.
template <int O, int I> kda_status spans_ok(const Span (&outs)[O], const Span (&ins)[I]) {
    for (const Span &s : outs)
        if (reinterpret_cast<uintptr_t>(s.p) % s.align) return KDA_ERR_ALIGN;
    for (const Span &s : ins)
        if (reinterpret_cast<uintptr_t>(s.p) % s.align) return KDA_ERR_ALIGN;
    for (int i = 0; i < O; ++i) {
        for (const Span &s : ins)
            if (overlap(outs[i].p, outs[i].n, s.p, s.n)) return KDA_ERR_ALIAS;
        for (int j = 0; j < i; ++j)
            if (overlap(outs[i].p, outs[i].n, outs[j].p, outs[j].n)) return KDA_ERR_ALIAS;
    }
    return KDA_OK;
}

int shift_of(int block_size) {
    for (int s = 4; s <= 7; ++s)
        if (block_size == 1 << s) return s;
    return -1;
}

// At most 2^30 tokens a row: positions stay within 32 bits.
bool reach_ok(long max_blocks, int shift) { return max_blocks << shift <= 1L << 30; }

kda_status check_pages(const kda_pages_desc *d, PagesArgs &a, bool table) {
    if (!d) return KDA_ERR_NULL;
    if (d->num_seqs < 0 || d->total_tokens < 0 || d->rows <= 0 || (table && (d->max_blocks <= 0 || d->num_free < 0))) return KDA_ERR_SHAPE;
    const int shift = shift_of(d->block_size);
    if (shift < 0 || (table && !reach_ok(d->max_blocks, shift))) return KDA_ERR_UNSUPPORTED;
    a = PagesArgs{};
    a.num_seqs = d->num_seqs;
    a.total_tokens = d->total_tokens;
    a.rows = d->rows;
    a.max_blocks = d->max_blocks;
    a.block_shift = shift;
    a.num_free = d->num_free;
    return KDA_OK;
}

kda_status check_kv(const kda_kv_desc *d, bool attend) {
    if (!d) return KDA_ERR_NULL;
    if (d->total_tokens < 0 || d->kv_heads <= 0 || d->num_blocks <= 0) return KDA_ERR_SHAPE;
    const int shift = shift_of(d->block_size);
    if ((d->head_dim != 64 && d->head_dim != 128) || shift < 0 || !dtype_ok(d->io_dtype)) return KDA_ERR_UNSUPPORTED;
    if (((long)d->num_blocks << shift) > INT32_MAX) return KDA_ERR_UNSUPPORTED;
    const long vec = d->io_dtype == KDA_BF16 ? 8 : 4, row = (long)d->kv_heads * d->head_dim;
    if (attend) {
        if (d->num_seqs < 0 || d->rows <= 0 || d->max_blocks <= 0 || d->q_heads <= 0 || d->q_heads % d->kv_heads != 0 ||
            d->q_stride < (long)d->q_heads * d->head_dim || !(d->scale > 0.f))
            return KDA_ERR_SHAPE;
        if (!reach_ok(d->max_blocks, shift) || !(d->scale <= 1048576.f) || (long)d->total_tokens * d->q_heads > INT32_MAX)
            return KDA_ERR_UNSUPPORTED;
        if (d->total_tokens > 1 && d->q_stride % vec) return KDA_ERR_ALIGN;
    } else {
        if (d->k_stride < row || d->v_stride < row) return KDA_ERR_SHAPE;
        if (d->kv_heads > 65535) return KDA_ERR_UNSUPPORTED;
        if (d->total_tokens > 1 && (d->k_stride % vec || d->v_stride % vec)) return KDA_ERR_ALIGN;
    }
    return KDA_OK;
}

kda_status check_sample(const kda_sample_desc *d) {
    if (!d) return KDA_ERR_NULL;
    if (d->num_rows < 0 || d->vocab <= 0 || d->stride < d->vocab) return KDA_ERR_SHAPE;
    if (!dtype_ok(d->logits_dtype) || d->vocab > (1 << 20)) return KDA_ERR_UNSUPPORTED;
    return d->num_rows == 0 || sample_fits(d->num_rows, d->vocab) ? KDA_OK : KDA_ERR_UNSUPPORTED;
}

}  // namespace

extern "C" {

kda_status kda_kv_reserve(const kda_pages_desc *d, const int32_t *cu_seqlens, const int32_t *state_indices,
                          const int32_t *kv_lens, int32_t *blocks_held, int32_t *block_table,
                          const int32_t *free_blocks, int32_t *free_count, int32_t *slots, int32_t *kv_totals,
                          void *stream) {
    PagesArgs a;
    const kda_status st = check_pages(d, a, true);
    if (st != KDA_OK) return st;
    const size_t N = d->num_seqs, T = d->total_tokens;
    if (N == 0 && T == 0) return KDA_OK;
    if (!free_count || (T && !slots) || (N && (!cu_seqlens || !state_indices || !kv_lens || !blocks_held || !block_table || !kv_totals)) ||
        (d->num_free && !free_blocks))
        return KDA_ERR_NULL;
    const Span outs[] = {{blocks_held, (size_t)d->rows * 4, 4}, {block_table, (size_t)d->rows * d->max_blocks * 4, 4}, {free_count, 4, 4},
                         {slots, T * 4, 4}, {kv_totals, N * 4, 4}};
    const Span ins[] = {{cu_seqlens, N ? (N + 1) * 4 : 0, 4}, {state_indices, N * 4, 4}, {kv_lens, (size_t)d->rows * 4, 4},
                        {free_blocks, (size_t)d->num_free * 4, 4}};
    const kda_status ss = spans_ok(outs, ins);
    if (ss != KDA_OK) return ss;
    a.cu_seqlens = cu_seqlens; a.indices = state_indices;
    a.kv_lens = const_cast<int32_t *>(kv_lens);
    a.blocks_held = blocks_held; a.block_table = block_table;
    a.free_blocks = const_cast<int32_t *>(free_blocks);
    a.free_count = free_count; a.slots = slots; a.kv_totals = kv_totals;
    return hip_status(launch_reserve(a, static_cast<hipStream_t>(stream)));
}

kda_status kda_kv_commit(const kda_pages_desc *d, const int32_t *cu_seqlens, const int32_t *steps,
                         const int32_t *state_indices, int32_t *kv_lens, const int32_t *blocks_held, void *stream) {
    PagesArgs a;
    const kda_status st = check_pages(d, a, false);
    if (st != KDA_OK) return st;
    const size_t N = d->num_seqs;
    if (N == 0) return KDA_OK;
    if (!cu_seqlens || !state_indices || !kv_lens || !blocks_held) return KDA_ERR_NULL;
    const Span outs[] = {{kv_lens, (size_t)d->rows * 4, 4}};
    const Span ins[] = {{cu_seqlens, (N + 1) * 4, 4}, {steps, steps ? N * 4 : 0, 4}, {state_indices, N * 4, 4}, {blocks_held, (size_t)d->rows * 4, 4}};
    const kda_status ss = spans_ok(outs, ins);
    if (ss != KDA_OK) return ss;
    a.cu_seqlens = cu_seqlens; a.indices = state_indices; a.steps = steps;
    a.kv_lens = kv_lens;
    a.blocks_held = const_cast<int32_t *>(blocks_held);
    return hip_status(launch_kv_commit(a, static_cast<hipStream_t>(stream)));
}

kda_status kda_kv_release(const kda_pages_desc *d, const int32_t *keep_lens, const int32_t *state_indices,
                          int32_t *kv_lens, int32_t *blocks_held, const int32_t *block_table, int32_t *free_blocks,
                          int32_t *free_count, void *stream) {
    PagesArgs a;
    const kda_status st = check_pages(d, a, true);
    if (st != KDA_OK) return st;
    const size_t N = d->num_seqs;
    if (N == 0) return KDA_OK;
    if (!state_indices || !kv_lens || !blocks_held || !block_table || !free_count || (d->num_free && !free_blocks)) return KDA_ERR_NULL;
    const Span outs[] = {{kv_lens, (size_t)d->rows * 4, 4}, {blocks_held, (size_t)d->rows * 4, 4}, {free_blocks, (size_t)d->num_free * 4, 4},
                         {free_count, 4, 4}};
    const Span ins[] = {{keep_lens, keep_lens ? N * 4 : 0, 4}, {state_indices, N * 4, 4}, {block_table, (size_t)d->rows * d->max_blocks * 4, 4}};
    const kda_status ss = spans_ok(outs, ins);
    if (ss != KDA_OK) return ss;
    a.indices = state_indices; a.keep_lens = keep_lens;
    a.kv_lens = kv_lens; a.blocks_held = blocks_held;
    a.block_table = const_cast<int32_t *>(block_table);
    a.free_blocks = free_blocks; a.free_count = free_count;
    return hip_status(launch_release(a, static_cast<hipStream_t>(stream)));
}

kda_status kda_kv_store(const kda_kv_desc *d, const void *k, const void *v, const int32_t *slots, void *k_cache,
                        void *v_cache, float *k_scale, float *v_scale, void *stream) {
    const kda_status st = check_kv(d, false);
    if (st != KDA_OK) return st;
    const long T = d->total_tokens;
    if (T == 0) return KDA_OK;
    if (!k || !v || !slots || !k_cache || !v_cache || !k_scale || !v_scale) return KDA_ERR_NULL;
    const long row = (long)d->kv_heads * d->head_dim;
    const size_t isz = io_size(d->io_dtype), cache = (size_t)d->num_blocks * d->block_size * row, scales = (size_t)d->num_blocks * d->kv_heads * 4;
    const Span outs[] = {{k_cache, cache, 16}, {v_cache, cache, 16}, {k_scale, scales, 4}, {v_scale, scales, 4}};
    const Span ins[] = {{k, rows_bytes(T, d->k_stride, row, isz), 16}, {v, rows_bytes(T, d->v_stride, row, isz), 16}, {slots, (size_t)T * 4, 4}};
    const kda_status ss = spans_ok(outs, ins);
    if (ss != KDA_OK) return ss;
    StoreArgs a{};
    a.k = k; a.v = v; a.slots = slots;
    a.k_cache = static_cast<uint8_t *>(k_cache);
    a.v_cache = static_cast<uint8_t *>(v_cache);
    a.k_scale = k_scale; a.v_scale = v_scale;
    a.total_tokens = d->total_tokens; a.heads = d->kv_heads; a.d = d->head_dim;
    a.block_shift = shift_of(d->block_size);
    a.num_blocks = d->num_blocks;
    a.io_bf16 = d->io_dtype == KDA_BF16;
    a.k_stride = d->k_stride; a.v_stride = d->v_stride;
    return hip_status(launch_kv_store(a, static_cast<hipStream_t>(stream)));
}

size_t kda_kv_attention_workspace_size(const kda_kv_desc *d) {
    if (check_kv(d, true) != KDA_OK || d->total_tokens == 0 || d->num_seqs == 0) return 0;
    return attend_workspace_bytes(d->num_seqs, d->total_tokens, d->q_heads, d->kv_heads, d->head_dim, d->io_dtype == KDA_BF16);
}

kda_status kda_kv_attention(const kda_kv_desc *d, const void *q, const int32_t *cu_seqlens, const int32_t *kv_totals,
                            const int32_t *state_indices, const int32_t *block_table, const void *k_cache,
                            const void *v_cache, const float *k_scale, const float *v_scale, void *o, void *workspace,
                            size_t workspace_bytes, void *stream) {
    const kda_status st = check_kv(d, true);
    if (st != KDA_OK) return st;
    const long T = d->total_tokens;
    const size_t N = d->num_seqs;
    if (T == 0 || N == 0) return KDA_OK;
    if (!q || !cu_seqlens || !kv_totals || !state_indices || !block_table || !k_cache || !v_cache || !k_scale || !v_scale || !o)
        return KDA_ERR_NULL;
    const size_t need = kda_kv_attention_workspace_size(d);
    if (need && (!workspace || workspace_bytes < need)) return KDA_ERR_WORKSPACE;
    const long qrow = (long)d->q_heads * d->head_dim, row = (long)d->kv_heads * d->head_dim;
    const size_t isz = io_size(d->io_dtype), cache = (size_t)d->num_blocks * d->block_size * row, scales = (size_t)d->num_blocks * d->kv_heads * 4;
    const Span outs[] = {{o, (size_t)T * qrow * isz, 16}, {workspace, need, 16}};
    const Span ins[] = {{q, rows_bytes(T, d->q_stride, qrow, isz), 16}, {cu_seqlens, (N + 1) * 4, 4}, {kv_totals, N * 4, 4},
                        {state_indices, N * 4, 4}, {block_table, (size_t)d->rows * d->max_blocks * 4, 4}, {k_cache, cache, 16},
                        {v_cache, cache, 16}, {k_scale, scales, 4}, {v_scale, scales, 4}};
    const kda_status ss = spans_ok(outs, ins);
    if (ss != KDA_OK) return ss;
    if (attend_grid(d->num_seqs, d->total_tokens, d->q_heads, d->kv_heads, d->head_dim, d->io_dtype == KDA_BF16) > INT32_MAX / 256)
        return KDA_ERR_UNSUPPORTED;
    AttendArgs a{};
    a.q = q; a.cu_seqlens = cu_seqlens; a.kv_totals = kv_totals; a.indices = state_indices; a.block_table = block_table;
    a.k_cache = static_cast<const uint8_t *>(k_cache);
    a.v_cache = static_cast<const uint8_t *>(v_cache);
    a.k_scale = k_scale; a.v_scale = v_scale;
    a.o = o;
    a.num_seqs = d->num_seqs; a.total_tokens = d->total_tokens; a.q_heads = d->q_heads; a.heads = d->kv_heads; a.d = d->head_dim;
    a.block_shift = shift_of(d->block_size);
    a.num_blocks = d->num_blocks; a.rows = d->rows; a.max_blocks = d->max_blocks;
    a.io_bf16 = d->io_dtype == KDA_BF16;
    a.q_stride = d->q_stride;
    a.scale = d->scale;
    return hip_status(launch_attend(a, workspace, static_cast<hipStream_t>(stream)));
}

size_t kda_sample_tokens_workspace_size(const kda_sample_desc *d) {
    if (check_sample(d) != KDA_OK || d->num_rows == 0) return 0;
    return sample_workspace_bytes(d->num_rows, d->vocab);
}

kda_status kda_sample_tokens(const kda_sample_desc *d, const void *logits, const float *uniform, const float *temperature,
                             const int32_t *top_k, const float *top_p, const float *min_p, int32_t *tokens, float *probs,
                             void *workspace, size_t workspace_bytes, void *stream) {
    const kda_status st = check_sample(d);
    if (st != KDA_OK) return st;
    const size_t N = d->num_rows, V = d->vocab;
    if (N == 0) return KDA_OK;
    if (!logits || (!tokens && !probs) || (tokens && !uniform)) return KDA_ERR_NULL;
    const size_t need = kda_sample_tokens_workspace_size(d), isz = io_size(d->logits_dtype);
    if (need && (!workspace || workspace_bytes < need)) return KDA_ERR_WORKSPACE;
    const Span outs[] = {{tokens, tokens ? N * 4 : 0, 4}, {probs, probs ? N * V * 4 : 0, 4}, {workspace, need, 16}};
    const Span ins[] = {{logits, rows_bytes(d->num_rows, d->stride, d->vocab, isz), (unsigned)isz}, {uniform, uniform ? N * 4 : 0, 4},
                        {temperature, temperature ? N * 4 : 0, 4}, {top_k, top_k ? N * 4 : 0, 4}, {top_p, top_p ? N * 4 : 0, 4},
                        {min_p, min_p ? N * 4 : 0, 4}};
    const kda_status ss = spans_ok(outs, ins);
    if (ss != KDA_OK) return ss;
    SampleArgs a{};
    a.logits = logits; a.uniform = uniform; a.temperature = temperature; a.top_p = top_p; a.min_p = min_p; a.top_k = top_k;
    a.tokens = tokens; a.probs = probs;
    a.rows = d->num_rows; a.vocab = d->vocab;
    a.bf16 = d->logits_dtype == KDA_BF16;
    a.stride = d->stride;
    return hip_status(launch_sample(a, workspace, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
