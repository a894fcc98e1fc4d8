"""GB300-native block-quantized weight-only matmul (MatMulNBits INT4/INT3) and
the QMoE expert FFN built on it, with the paged key-value cache (16-bit or 8-bit
codes), the plan of its pages, the attention over it, the token probabilities and
the draft verification that a decoder needs around them.

The compute lives in the CUDA library ``_build/libmnb.so`` (hand-written
sm_103a kernels behind the C ABI of ``include/mnb.h``); this package is its
thin ctypes binding.  Build it with ``__graft_entry__.build()`` or
``python -m qmoe_mnb_matmul_gb300._build``.
"""
from ._binding import (BF16, E4M3, F16, F32, FC1_CONCAT, FC1_INTERLEAVED, KvCacheDesc, KvPoolDesc,  # noqa: F401
                       KvRopeDesc, KvStepDesc, MnbError, PrepackedDesc, QmoeOptions, TokenRules, draft_verify,
                       header_functions, kv_append, kv_attention, kv_attention_workspace_size, kv_cache, kv_plan,
                       kv_pool, kv_rope, kv_step, library_path,
                       load_library, mnb_diag_wait_timeout, mnb_gate_up_swiglu, mnb_get_last_device_error, mnb_matmul, mnb_matmul_int8a,
                       mnb_matmul_prepacked, mnb_matmul_workspace_size, mnb_pack_codes, mnb_prepack,
                       mnb_prepack_size, mnb_quantize_int3, mnb_status_string, mnb_unpack_codes, mnb_validate_host,
                       qmoe_forward, qmoe_forward_ex, qmoe_forward_static, qmoe_permute, qmoe_route,
                       qmoe_workspace_size, token_probs, token_rules)

__all__ = ["mnb_matmul", "mnb_matmul_int8a", "mnb_gate_up_swiglu", "mnb_matmul_workspace_size", "mnb_prepack",
           "mnb_prepack_size", "mnb_matmul_prepacked", "PrepackedDesc", "qmoe_forward", "qmoe_forward_ex",
           "qmoe_forward_static", "qmoe_workspace_size", "qmoe_route", "qmoe_permute", "QmoeOptions",
           "kv_cache", "kv_step", "kv_rope", "kv_append", "kv_attention", "kv_attention_workspace_size",
           "kv_pool", "kv_plan", "token_rules", "token_probs",
           "draft_verify", "KvCacheDesc", "KvStepDesc", "KvRopeDesc", "KvPoolDesc", "TokenRules", "mnb_unpack_codes",
           "mnb_pack_codes", "mnb_quantize_int3", "mnb_validate_host",
           "mnb_get_last_device_error", "mnb_diag_wait_timeout", "mnb_status_string", "load_library",
           "library_path", "MnbError"]
