// Paged attention over 8-bit codes, fp32 queries, heads of up to 96 (see kv_attention8_impl.cuh).
#include "kv_attention8_impl.cuh"

namespace mnb {
MNB_KV_ATTENTION8_SLICE(kv_attention8_qf32_96, true, 96)
}  // namespace mnb
