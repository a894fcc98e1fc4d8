// kv_api.cu -- the extern "C" entry points of the paged key-value cache, its plan,
// the token probabilities and the draft verification: host-side metadata validation (payloads are never read
// on the host) and launches on the caller's stream.
#include <cmath>

#include "api_util.h"
#include "common.cuh"
#include "kernels.h"
#include "kv.h"

namespace mnb {

namespace {

constexpr int64_t kMaxInt = (int64_t(1) << 31) - 1;

// The largest element offset of a strided array stays below 2^61.
bool span_ok(int64_t extent, int64_t stride, int64_t* total) {
    int64_t n;
    return mul_ok(extent, stride, &n) && mul_ok(n, 4, &n) && (*total += n) < (int64_t(1) << 62);
}

mnb_status check_cache(const kv_cache_desc* d, KvCache* c) {
    if (!d || !d->k || !d->v) return MNB_ERR_INVALID_ARG;
    const bool codes = d->dtype == MNB_E4M3;
    if (d->num_pages < 1 || d->page_size < 1 || d->kv_heads < 1 || d->head_dim < 1 || !(valid_dtype(d->dtype) || codes))
        return MNB_ERR_INVALID_ARG;
    if (d->dtype == MNB_F32) return MNB_ERR_UNSUPPORTED;
    if (d->head_dim % 8 || d->head_dim < 16 || d->head_dim > 256 || d->page_size % 8) return MNB_ERR_UNSUPPORTED;
    c->k = d->k;
    c->v = d->v;
    c->num_pages = d->num_pages;
    c->page_size = d->page_size;
    c->heads = d->kv_heads;
    c->dim = d->head_dim;
    c->dtype = d->dtype;
    c->token_stride = d->token_stride;
    // the stride of an extent of one is never used
    c->head_stride = d->kv_heads > 1 ? d->head_stride : d->head_dim;
    c->page_stride = d->num_pages > 1 ? d->page_stride : d->head_dim;
    for (const int64_t s : {c->token_stride, c->head_stride, c->page_stride}) {
        if (s < c->dim) return MNB_ERR_INVALID_ARG;
        if (s % (codes ? 16 : 8) || s >= (int64_t(1) << 38)) return MNB_ERR_UNSUPPORTED;  // whole 16-byte units, below 2^40 bytes
    }
    if (!aligned(d->k, 16) || !aligned(d->v, 16)) return MNB_ERR_UNSUPPORTED;
    if (codes) {
        if (!d->k_scale || !d->v_scale || d->scale_block < 1) return MNB_ERR_INVALID_ARG;
        if (d->head_dim % 16 || d->scale_block < 8 || d->scale_block > 128 || (d->scale_block & (d->scale_block - 1)) ||
            d->page_size % d->scale_block || !aligned(d->k_scale, 4) || !aligned(d->v_scale, 4))
            return MNB_ERR_UNSUPPORTED;
        const int64_t blocks = d->page_size / d->scale_block;
        c->k_scale = d->k_scale;
        c->v_scale = d->v_scale;
        c->scale_head_stride = d->kv_heads > 1 ? d->scale_head_stride : blocks;
        c->scale_page_stride = d->num_pages > 1 ? d->scale_page_stride : blocks;
        c->block_shift = 0;
        while ((1 << c->block_shift) < d->scale_block) ++c->block_shift;
        int64_t span = 0;
        for (const int64_t s : {c->scale_head_stride, c->scale_page_stride})
            if (s < blocks) return MNB_ERR_INVALID_ARG;
        if (!span_ok(c->num_pages, c->scale_page_stride, &span) || !span_ok(c->heads, c->scale_head_stride, &span))
            return MNB_ERR_SIZE_OVERFLOW;
    }
    int64_t total = 0;
    if (!span_ok(c->num_pages, c->page_stride, &total) || !span_ok(c->heads, c->head_stride, &total) ||
        !span_ok(c->page_size, c->token_stride, &total))
        return MNB_ERR_SIZE_OVERFLOW;
    if (c->num_pages > kMaxInt) return MNB_ERR_SIZE_OVERFLOW;
    return MNB_OK;
}

// `nothing`: the step has no token, so that the call has nothing to do.
mnb_status check_step(const kv_step_desc* d, const KvCache& c, KvStep* s, bool* nothing) {
    *nothing = false;
    if (!d || d->batch < 0 || d->tokens < 0 || d->max_new < 1) return MNB_ERR_INVALID_ARG;
    if (d->batch == 0 || d->tokens == 0) {
        *nothing = true;
        return MNB_OK;
    }
    if (!d->seq_lens || !d->page_table || d->max_pages < 1 || d->table_stride < d->max_pages) return MNB_ERR_INVALID_ARG;
    if (!d->new_start && d->tokens != d->batch) return MNB_ERR_INVALID_ARG;
    if (d->tokens > (1 << 30)) return MNB_ERR_SIZE_OVERFLOW;  // token and row numbers are 32-bit
    if (!aligned(d->seq_lens, 4) || !aligned(d->new_start, 4) || !aligned(d->page_table, 4)) return MNB_ERR_UNSUPPORTED;
    int64_t total = 0;
    if (!span_ok(d->batch, d->table_stride, &total)) return MNB_ERR_SIZE_OVERFLOW;
    s->seq_lens = d->seq_lens;
    s->new_start = d->new_start;
    s->page_table = d->page_table;
    s->table_stride = d->table_stride;
    s->batch = d->batch;
    s->tokens = d->tokens;
    s->max_pages = d->max_pages;
    const int64_t cap = int64_t(d->max_pages) * c.page_size;
    s->capacity = static_cast<int>(cap < kKvMaxCapacity ? cap : kKvMaxCapacity);
    return MNB_OK;
}

// One of q, k, v or an output: [tokens, heads, dim] with `stride` elements
// between tokens, read and written in 16-byte units.
mnb_status check_rows(const void* p, int64_t stride, int64_t heads, int64_t dim, int64_t tokens) {
    if (stride < heads * dim) return MNB_ERR_INVALID_ARG;
    if (!aligned(p, 16) || stride % 8) return MNB_ERR_UNSUPPORTED;
    int64_t total = 0;
    return span_ok(tokens, stride, &total) ? MNB_OK : MNB_ERR_SIZE_OVERFLOW;
}

}  // namespace
}  // namespace mnb

using namespace mnb;

extern "C" {

mnb_status kv_append(const kv_cache_desc* cache, const kv_step_desc* step, const kv_rope_desc* rope, const void* q,
                     int64_t q_stride, int64_t q_heads, const void* k, int64_t k_stride, const void* v,
                     int64_t v_stride, mnb_dtype dtype, void* q_out, int64_t q_out_stride, mnb_stream_t stream) {
    KvAppendArgs a = {};
    mnb_status st = check_cache(cache, &a.cache);
    if (st != MNB_OK) return st;
    bool nothing;
    if ((st = check_step(step, a.cache, &a.step, &nothing)) != MNB_OK) return st;
    if (!valid_dtype(dtype) || (q == nullptr) != (q_out == nullptr) || (q && q_heads < 1)) return MNB_ERR_INVALID_ARG;
    if (dtype != MNB_F32 && dtype != a.cache.dtype && a.cache.dtype != MNB_E4M3) return MNB_ERR_UNSUPPORTED;
    if (rope) {
        if (rope->cos_sin) {
            if (rope->max_pos < 1 || rope->rot_dim < 1 || rope->rot_dim > a.cache.dim) return MNB_ERR_INVALID_ARG;
            if (rope->rot_dim % 8) return MNB_ERR_UNSUPPORTED;
            int64_t total = 0;
            if (!span_ok(rope->max_pos, rope->rot_dim, &total)) return MNB_ERR_SIZE_OVERFLOW;
        }
        if ((rope->q_norm || rope->k_norm) && !(rope->eps >= 0.f && std::isfinite(rope->eps))) return MNB_ERR_INVALID_ARG;
        if (!aligned(rope->cos_sin, 16) || !aligned(rope->q_norm, 16) || !aligned(rope->k_norm, 16))
            return MNB_ERR_UNSUPPORTED;
        a.cos_sin = rope->cos_sin;
        a.max_pos = rope->max_pos;
        a.rot_dim = rope->cos_sin ? rope->rot_dim : 0;
        a.interleaved = rope->interleaved != 0;
        a.q_norm = rope->q_norm;
        a.k_norm = rope->k_norm;
        a.eps = rope->eps;
    }
    if (nothing) return MNB_OK;
    if (!k || !v) return MNB_ERR_INVALID_ARG;
    if (q && q_heads > kMaxInt / (a.cache.dim * 4)) return MNB_ERR_SIZE_OVERFLOW;
    if ((st = check_rows(k, k_stride, a.cache.heads, a.cache.dim, a.step.tokens)) != MNB_OK) return st;
    if ((st = check_rows(v, v_stride, a.cache.heads, a.cache.dim, a.step.tokens)) != MNB_OK) return st;
    if (q) {
        if ((st = check_rows(q, q_stride, q_heads, a.cache.dim, a.step.tokens)) != MNB_OK) return st;
        if ((st = check_rows(q_out, q_out_stride, q_heads, a.cache.dim, a.step.tokens)) != MNB_OK) return st;
    }
    a.q = q;
    a.k = k;
    a.v = v;
    a.q_stride = q_stride;
    a.k_stride = k_stride;
    a.v_stride = v_stride;
    a.q_heads = q ? static_cast<int>(q_heads) : 0;
    a.in_dtype = dtype;
    a.q_out = q_out;
    a.q_out_stride = q_out_stride;
    const int sms = sm_count_current();
    if (sms <= 0) return MNB_ERR_CUDA;
    auto launch = a.cache.dtype == MNB_E4M3 ? launch_kv_append8 : launch_kv_append;
    return from_cuda(launch(a, sms, pdl_enabled(), reinterpret_cast<cudaStream_t>(stream)));
}

mnb_status kv_attention_workspace_size(int64_t q_heads, int64_t kv_heads, int64_t head_dim, int64_t max_new,
                                       size_t* bytes) {
    if (!bytes) return MNB_ERR_INVALID_ARG;
    *bytes = 0;
    if (q_heads < 1 || kv_heads < 1 || q_heads % kv_heads || head_dim < 1 || max_new < 1) return MNB_ERR_INVALID_ARG;
    if (head_dim % 8 || head_dim < 16 || head_dim > 256) return MNB_ERR_UNSUPPORTED;
    if (q_heads > kMaxInt || max_new > kMaxInt) return MNB_ERR_SIZE_OVERFLOW;
    const int rows = kv_attention_rows(static_cast<int>(q_heads / kv_heads), max_new);
    *bytes = static_cast<size_t>(kv_attention_space(rows, kv_attention_pad(static_cast<int>(head_dim))).total);
    return MNB_OK;
}

mnb_status kv_attention(const kv_cache_desc* cache, const kv_step_desc* step, const void* q, int64_t q_stride,
                        int64_t q_heads, mnb_dtype dtype, void* out, int64_t out_stride, float* lse, float scale,
                        int64_t window, void* workspace, size_t workspace_bytes, mnb_stream_t stream) {
    KvAttnArgs a = {};
    mnb_status st = check_cache(cache, &a.cache);
    if (st != MNB_OK) return st;
    bool nothing;
    if ((st = check_step(step, a.cache, &a.step, &nothing)) != MNB_OK) return st;
    if (!valid_dtype(dtype) || q_heads < 1 || q_heads % a.cache.heads || window < 0 ||
        !(scale > 0.f && std::isfinite(scale)))
        return MNB_ERR_INVALID_ARG;
    if (dtype != MNB_F32 && dtype != a.cache.dtype && a.cache.dtype != MNB_E4M3) return MNB_ERR_UNSUPPORTED;
    if (nothing) return MNB_OK;
    if (!q || !out) return MNB_ERR_INVALID_ARG;
    if (q_heads > kMaxInt / (a.cache.dim * 4) || step->tokens > (int64_t(1) << 30) / q_heads) return MNB_ERR_SIZE_OVERFLOW;
    if ((st = check_rows(q, q_stride, q_heads, a.cache.dim, a.step.tokens)) != MNB_OK) return st;
    if ((st = check_rows(out, out_stride, q_heads, a.cache.dim, a.step.tokens)) != MNB_OK) return st;
    if (!aligned(lse, 4)) return MNB_ERR_UNSUPPORTED;
    a.group = static_cast<int>(q_heads / a.cache.heads);
    const int rows = kv_attention_rows(a.group, step->max_new);
    if (!workspace || int64_t(workspace_bytes) < kv_attention_space(rows, kv_attention_pad(a.cache.dim)).total)
        return MNB_ERR_WORKSPACE;
    if (!aligned(workspace, 256)) return MNB_ERR_UNSUPPORTED;
    a.q = q;
    a.q_stride = q_stride;
    a.out = out;
    a.out_stride = out_stride;
    a.lse = lse;
    a.scale = scale;
    a.window = static_cast<int>(window <= kMaxInt ? window : 0);  // positions are 32-bit: a wider one masks nothing
    const int sms = sm_count_current();
    if (sms <= 0) return MNB_ERR_CUDA;
    return from_cuda(launch_kv_attention(a, dtype, step->max_new, workspace, sms, pdl_enabled(),
                                         reinterpret_cast<cudaStream_t>(stream)));
}

mnb_status kv_plan(const kv_pool_desc* pool, const int32_t* keep, const int32_t* add, int32_t* seq_lens,
                   int32_t* new_start, int64_t max_tokens, int64_t* slots, int32_t* refused, mnb_stream_t stream) {
    if (!pool || pool->batch < 0 || pool->num_pages < 0 || pool->page_size < 1 || max_tokens < 0)
        return MNB_ERR_INVALID_ARG;
    if (!pool->free_count || !pool->free_count_out || !new_start || (pool->num_pages > 0 && !pool->free_pages))
        return MNB_ERR_INVALID_ARG;
    if (pool->batch > 0 && (!pool->held || !pool->held_out || !pool->page_table || !keep || !add || !seq_lens ||
                            pool->max_pages < 1 || pool->table_stride < pool->max_pages))
        return MNB_ERR_INVALID_ARG;
    if (pool->batch > kKvPlanMaxBatch) return MNB_ERR_UNSUPPORTED;
    if (max_tokens > (int64_t(1) << 30)) return MNB_ERR_SIZE_OVERFLOW;
    for (const void* p : {static_cast<const void*>(pool->held), static_cast<const void*>(pool->page_table),
                          static_cast<const void*>(pool->free_pages), static_cast<const void*>(pool->free_count),
                          static_cast<const void*>(pool->held_out), static_cast<const void*>(pool->free_count_out),
                          static_cast<const void*>(keep), static_cast<const void*>(add),
                          static_cast<const void*>(seq_lens), static_cast<const void*>(new_start),
                          static_cast<const void*>(refused)})
        if (!aligned(p, 4)) return MNB_ERR_UNSUPPORTED;
    if (!aligned(slots, 8)) return MNB_ERR_UNSUPPORTED;
    int64_t total = 0;
    if (!span_ok(pool->batch, pool->table_stride, &total)) return MNB_ERR_SIZE_OVERFLOW;
    KvPlanArgs a = {};
    a.held = pool->held;
    a.keep = keep;
    a.add = add;
    a.free_count = pool->free_count;
    a.page_table = pool->page_table;
    a.table_stride = pool->table_stride;
    a.free_pages = pool->free_pages;
    a.batch = pool->batch;
    a.max_pages = pool->max_pages;
    a.page_size = pool->page_size;
    a.num_pages = pool->num_pages;
    a.max_tokens = static_cast<uint32_t>(max_tokens);
    a.held_out = pool->held_out;
    a.free_count_out = pool->free_count_out;
    a.seq_lens = seq_lens;
    a.new_start = new_start;
    a.refused = refused;
    a.slots = slots;
    const int sms = sm_count_current();
    if (sms <= 0) return MNB_ERR_CUDA;
    return from_cuda(launch_kv_plan(a, sms, pdl_enabled(), reinterpret_cast<cudaStream_t>(stream)));
}

mnb_status token_probs(const void* logits, mnb_dtype dtype, int64_t logits_seq_stride, int64_t logits_row_stride,
                       const int32_t* row_start, int64_t tokens, const token_rules* rules,
                       const int32_t* draft_tokens, const uint32_t* mask, int64_t mask_seq_stride,
                       int64_t mask_row_stride, int64_t rows, int64_t vocab, float* out, int64_t out_seq_stride,
                       int64_t out_row_stride, int softmax, mnb_stream_t stream) {
    if (!rules || !valid_dtype(dtype) || rules->batch < 0 || rows < 0 || vocab < 1 || rules->history_columns < 0 ||
        rules->biases < 0 || tokens < 0)
        return MNB_ERR_INVALID_ARG;
    const int64_t batch = rules->batch;
    if (batch == 0 || rows == 0) return MNB_OK;
    if ((!logits && !(row_start && tokens == 0)) || !out) return MNB_ERR_INVALID_ARG;
    if (rules->history && (!rules->history_lens || rules->history_stride < rules->history_columns)) return MNB_ERR_INVALID_ARG;
    if (rules->biases > 0 && (!rules->bias_tokens || !rules->bias_values || rules->bias_stride < rules->biases))
        return MNB_ERR_INVALID_ARG;
    // rows that are only read may be shared
    if (logits_row_stride < 0 || logits_seq_stride < 0 || mask_seq_stride < 0 || mask_row_stride < 0) return MNB_ERR_INVALID_ARG;
    if ((rows > 1 && out_row_stride < vocab) || (batch > 1 && out_seq_stride < vocab)) return MNB_ERR_INVALID_ARG;
    if (vocab >= (int64_t(1) << 22) || rows > 1025) return MNB_ERR_UNSUPPORTED;
    const bool drafts = draft_tokens != nullptr && rows > 1;
    const int64_t listed = (rules->history ? rules->history_columns : 0) + (drafts ? rows - 1 : 0) + rules->biases;
    if (!token_probs_fits(vocab, listed)) return MNB_ERR_UNSUPPORTED;
    if ((rules->history ? rules->history_columns : 0) + rows > kProbMostHistory || rules->biases > kProbMostBiases)
        return MNB_ERR_UNSUPPORTED;
    if (batch * rows > kMaxInt / 16) return MNB_ERR_SIZE_OVERFLOW;
    for (const void* p : {static_cast<const void*>(row_start), static_cast<const void*>(rules->temperature),
                          static_cast<const void*>(rules->history), static_cast<const void*>(rules->history_lens),
                          static_cast<const void*>(rules->prompt_lens), static_cast<const void*>(rules->repetition),
                          static_cast<const void*>(rules->frequency), static_cast<const void*>(rules->presence),
                          static_cast<const void*>(rules->bias_tokens), static_cast<const void*>(rules->bias_values),
                          static_cast<const void*>(draft_tokens), static_cast<const void*>(mask),
                          static_cast<const void*>(out)})
        if (!aligned(p, 4)) return MNB_ERR_UNSUPPORTED;
    if (!aligned(logits, dsize(dtype))) return MNB_ERR_UNSUPPORTED;
    int64_t total = 0;
    if (row_start ? !span_ok(tokens, logits_row_stride, &total)
                  : !span_ok(batch, logits_seq_stride, &total) || !span_ok(rows, logits_row_stride, &total))
        return MNB_ERR_SIZE_OVERFLOW;
    total = 0;
    if (!span_ok(batch, out_seq_stride, &total) || !span_ok(rows, out_row_stride, &total)) return MNB_ERR_SIZE_OVERFLOW;
    total = 0;
    if (!span_ok(batch, mask_seq_stride, &total) || !span_ok(rows, mask_row_stride, &total)) return MNB_ERR_SIZE_OVERFLOW;
    total = 0;
    if (!span_ok(batch, rules->history_stride, &total) || !span_ok(batch, rules->bias_stride, &total))
        return MNB_ERR_SIZE_OVERFLOW;
    ProbArgs a = {};
    a.logits = logits;
    a.logits_seq = logits_seq_stride;
    a.logits_row = logits_row_stride;
    a.row_start = row_start;
    a.tokens = tokens;
    a.temperature = rules->temperature;
    a.repetition = rules->repetition;
    a.frequency = rules->frequency;
    a.presence = rules->presence;
    a.history = rules->history;
    a.history_stride = rules->history_stride;
    a.history_columns = rules->history_columns;
    a.history_lens = rules->history_lens;
    a.prompt_lens = rules->prompt_lens;
    a.bias_tokens = rules->bias_tokens;
    a.bias_values = rules->bias_values;
    a.bias_stride = rules->bias_stride;
    a.biases = rules->biases;
    a.draft_tokens = drafts ? draft_tokens : nullptr;
    a.mask = mask;
    a.mask_seq = mask_seq_stride;
    a.mask_row = mask_row_stride;
    a.batch = batch;
    a.vocab = vocab;
    a.rows = static_cast<int>(rows);
    a.out = out;
    a.out_seq = out_seq_stride;
    a.out_row = out_row_stride;
    a.softmax = softmax != 0;
    const int sms = sm_count_current();
    if (sms <= 0) return MNB_ERR_CUDA;
    return from_cuda(launch_token_probs(a, dtype, sms, pdl_enabled(), reinterpret_cast<cudaStream_t>(stream)));
}

mnb_status draft_verify(const float* target, int64_t target_seq_stride, int64_t target_row_stride, const float* draft,
                        int64_t draft_seq_stride, int64_t draft_row_stride, const int32_t* draft_tokens,
                        const int32_t* n_drafts, const float* uniforms, int64_t batch, int64_t drafts, int64_t vocab,
                        int32_t* tokens, int32_t* accepted, mnb_stream_t stream) {
    if (batch < 0 || drafts < 0 || vocab < 1) return MNB_ERR_INVALID_ARG;
    if (batch == 0) return MNB_OK;
    if (!target || !uniforms || !tokens || !accepted || (drafts > 0 && !draft_tokens)) return MNB_ERR_INVALID_ARG;
    // rows are only read: a stride of 0 shares one row among drafts or sequences
    if (target_row_stride < 0 || target_seq_stride < 0 || (draft && (draft_row_stride < 0 || draft_seq_stride < 0)))
        return MNB_ERR_INVALID_ARG;
    // fewer than 2^22 weights of at most 2^40 add up below 2^62
    if (vocab >= (int64_t(1) << 22) || drafts > 1024 || batch > kMaxInt / 16) return MNB_ERR_UNSUPPORTED;
    for (const void* p : {static_cast<const void*>(target), static_cast<const void*>(draft),
                          static_cast<const void*>(draft_tokens), static_cast<const void*>(n_drafts),
                          static_cast<const void*>(uniforms), static_cast<const void*>(tokens),
                          static_cast<const void*>(accepted)})
        if (!aligned(p, 4)) return MNB_ERR_UNSUPPORTED;
    int64_t total = 0;
    if (!span_ok(batch, target_seq_stride, &total) || !span_ok(drafts + 1, target_row_stride, &total))
        return MNB_ERR_SIZE_OVERFLOW;
    total = 0;
    if (draft && (!span_ok(batch, draft_seq_stride, &total) || !span_ok(drafts + 1, draft_row_stride, &total)))
        return MNB_ERR_SIZE_OVERFLOW;
    DraftArgs a = {};
    a.target = target;
    a.target_seq = target_seq_stride;
    a.target_row = target_row_stride;
    a.draft = drafts > 0 ? draft : nullptr;
    a.draft_seq = draft_seq_stride;
    a.draft_row = draft_row_stride;
    a.draft_tokens = draft_tokens;
    a.n_drafts = n_drafts;
    a.uniforms = uniforms;
    a.batch = batch;
    a.vocab = vocab;
    a.drafts = static_cast<int>(drafts);
    a.tokens = tokens;
    a.accepted = accepted;
    const int sms = sm_count_current();
    if (sms <= 0) return MNB_ERR_CUDA;
    return from_cuda(launch_draft_verify(a, sms, pdl_enabled(), reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
