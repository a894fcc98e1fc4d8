// Paged attention, bf16 cache and queries (see kv_attention_impl.cuh).
#include "kv_attention_impl.cuh"

namespace mnb {
MNB_KV_ATTENTION_SLICE(kv_attention_bf16, kBF16, false)
}  // namespace mnb
