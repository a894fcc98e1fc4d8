// Paged attention, fp16 cache and queries (see kv_attention_impl.cuh).
#include "kv_attention_impl.cuh"

namespace mnb {
MNB_KV_ATTENTION_SLICE(kv_attention_f16, kF16, false)
}  // namespace mnb
