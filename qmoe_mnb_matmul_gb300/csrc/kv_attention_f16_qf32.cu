// Paged attention, fp16 cache, fp32 queries (see kv_attention_impl.cuh).
#include "kv_attention_impl.cuh"

namespace mnb {
MNB_KV_ATTENTION_SLICE(kv_attention_f16_qf32, kF16, true)
}  // namespace mnb
