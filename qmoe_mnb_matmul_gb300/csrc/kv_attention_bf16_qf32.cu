// Paged attention, bf16 cache, fp32 queries (see kv_attention_impl.cuh).
#include "kv_attention_impl.cuh"

namespace mnb {
MNB_KV_ATTENTION_SLICE(kv_attention_bf16_qf32, kBF16, true)
}  // namespace mnb
