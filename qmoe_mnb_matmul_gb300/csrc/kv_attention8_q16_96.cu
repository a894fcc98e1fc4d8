// Paged attention over 8-bit codes, 16-bit queries, heads of up to 96 (see kv_attention8_impl.cuh).
#include "kv_attention8_impl.cuh"

namespace mnb {
MNB_KV_ATTENTION8_SLICE(kv_attention8_q16_96, false, 96)
}  // namespace mnb
