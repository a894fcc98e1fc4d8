// kv.h -- arguments and host-side launchers of the paged key-value cache
// kernels and of the draft verification (internal to the library).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/mnb.h"

namespace mnb {

// The paged cache: element (page, head, row in page, d) of keys or values is at
// page * page_stride + head * head_stride + row * token_stride + d.
struct KvCache {
    void* k;
    void* v;
    int64_t num_pages, page_stride, head_stride, token_stride;  // strides in elements
    int page_size, heads, dim, dtype;
};

// One step's tokens (device arrays of the caller).
struct KvStep {
    const int* seq_lens;    // [batch] tokens in the cache after the step
    const int* new_start;   // [batch + 1], or null: token b belongs to sequence b
    const int* page_table;  // [batch, max_pages], rows table_stride apart
    int64_t table_stride;
    int batch, tokens, max_pages;
    int capacity;           // min(max_pages * page_size, kKvMaxCapacity)
};
constexpr int kKvMaxCapacity = 0x7fffffff - 4096;  // positions are 32-bit, with room for a tile past the end

// First new token and number of new tokens of sequence b, kept inside
// [0, tokens] whatever new_start holds.
__device__ __forceinline__ void step_tokens(const KvStep& s, int b, int* first, int* count) {
    if (s.new_start == nullptr) {
        *first = b;
        *count = 1;
        return;
    }
    const int lo = min(max(__ldg(s.new_start + b), 0), s.tokens);
    const int hi = min(max(__ldg(s.new_start + b + 1), 0), s.tokens);
    *first = lo;
    *count = max(hi - lo, 0);
}

// ------------------------------------------------------------- kv_append

struct KvAppendArgs {
    KvCache cache;
    KvStep step;
    const void *q, *k, *v;
    int64_t q_stride, k_stride, v_stride;  // elements between tokens
    int q_heads, in_dtype;
    void* q_out;
    int64_t q_out_stride;
    const float* cos_sin;  // [max_pos, rot_dim]: rot_dim / 2 cosines, then as many sines; null: no rotation
    int64_t max_pos;
    int rot_dim, interleaved;
    const float *q_norm, *k_norm;  // [dim] or null
    float eps;
};
cudaError_t launch_kv_append(const KvAppendArgs& a, int sm_count, bool pdl, cudaStream_t stream);
cudaError_t kv_append_take_error(unsigned int* out);

// ---------------------------------------------------------- kv_attention

constexpr int kKvTile = 64;      // cached tokens per tile
constexpr int kKvMaxCtas = 304;  // CTAs of the main kernel: two on each of 152 SMs

// Division by a number fixed at launch: x / d = (hi32(x m) + x) >> s for 0 <= x < 2^31
// (Granlund and Montgomery, "Division by invariant integers using multiplication").
struct FastDiv {
    uint32_t m, s;
    void set(uint32_t d) {
        s = 0;
        while ((uint64_t(1) << s) < d) ++s;
        m = static_cast<uint32_t>(((uint64_t(1) << 32) * ((uint64_t(1) << s) - d)) / d + 1);
    }
#ifdef __CUDACC__
    __device__ __forceinline__ int operator()(int x) const {
        return static_cast<int>((__umulhi(static_cast<uint32_t>(x), m) + static_cast<uint32_t>(x)) >> s);
    }
#endif
};

// Attention weights are 2^(score - reference), where the reference is the row's largest
// score (in log2 units) less this shift: the range that the cache's type leaves free.
constexpr int kv_weight_shift(int dtype) { return dtype == MNB_F16 ? 15 : 0; }

#ifdef __CUDACC__
// Natural log-sum-exp of a row from its reference and its sum of weights.
__device__ __forceinline__ float kv_log_sum(float reference, float sum, int shift) {
    if (sum == 0.f) return -INFINITY;
    return (reference + shift + log2f(ldexpf(sum, -shift))) * 0.6931471805599453f;
}
#endif

struct KvAttnArgs {
    KvCache cache;
    KvStep step;
    const void* q;
    int64_t q_stride;
    void* out;
    int64_t out_stride;
    float* lse;  // [tokens, q_heads] or null
    int group;   // query heads per key-value head
    FastDiv by_group, by_page;  // division by group, by the page size
    float scale;
    int window;  // 0: every earlier token
    int box_rows;
    // partial results of the pairs split over CTAs: two slots per CTA
    float* part_o;     // [2 * ctas][rows][padded dim]
    float2* part_ml;   // [2 * ctas][rows]: reference, sum of weights
    // [ctas]: the pair that begins in this CTA and goes on in later ones: {last CTA (-1: no such
    // pair), 2 * rows + slot of its part here, first flat row (token * group + head in group), key-value head}
    int4* join;
};

// Rows of a row tile (8, 32 or 64) and the head dimension's padded width.
int kv_attention_rows(int group, int64_t max_new);
int kv_attention_pad(int dim);
struct KvAttnSpace {
    int64_t part_o, part_ml, join, total;  // byte offsets, bytes
};
KvAttnSpace kv_attention_space(int rows, int pad);
cudaError_t launch_kv_attention(const KvAttnArgs& a, int q_dtype, int64_t max_new, void* workspace, int sm_count,
                                bool pdl, cudaStream_t stream);
cudaError_t kv_attention_take_error(unsigned int* out);

// ---------------------------------------------------------- draft_verify

struct DraftArgs {
    const float* target;  // [batch][drafts + 1][vocab], sequence and row strides in elements
    int64_t target_seq, target_row;
    const float* draft;   // [batch][drafts][vocab] or null
    int64_t draft_seq, draft_row;
    const int* draft_tokens;  // [batch, drafts]
    const int* n_drafts;      // [batch] or null
    const float* uniforms;    // [batch, drafts + 1]
    int64_t batch, vocab;
    int drafts;
    int* tokens;              // [batch, drafts + 1]
    int* accepted;            // [batch]
};
cudaError_t launch_draft_verify(const DraftArgs& a, int sm_count, bool pdl, cudaStream_t stream);
cudaError_t draft_take_error(unsigned int* out);

}  // namespace mnb
