"""ctypes binding of libmnb.so: the C entry points of include/mnb.h under the
same names.  Argument marshalling only -- every step of every call runs in the
library's CUDA kernels.  There is no fallback: if the library has not been
built, loading it raises.

Tensors are torch tensors on the current CUDA device (contiguous); raw device
pointers may be passed as ints instead.  The paged-cache and draft calls take
tensors only, with strides where their text says so.  ``stream`` is a
torch.cuda.Stream, a raw cudaStream_t handle (int), or None for torch's current
stream.
"""
from __future__ import annotations

import ctypes
import os
import re

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
DEFAULT_LIB = os.path.join(HERE, "_build", "libmnb.so")
HEADER = os.path.join(ROOT, "include", "mnb.h")

STATUS = {0: "MNB_OK", 1: "MNB_ERR_INVALID_ARG", 2: "MNB_ERR_UNSUPPORTED", 3: "MNB_ERR_SIZE_OVERFLOW",
          4: "MNB_ERR_WORKSPACE", 5: "MNB_ERR_CUDA", 6: "MNB_ERR_TIMEOUT", 7: "MNB_ERR_CONTENT"}
F32, F16, BF16 = 0, 1, 2
E4M3 = 3  # of a key-value cache alone
FC1_INTERLEAVED, FC1_CONCAT = 0, 1


class PrepackedDesc(ctypes.Structure):
    """mnb_prepacked_desc: the host copy of a prepacked buffer's header."""
    _fields_ = [("magic", ctypes.c_uint32), ("version", ctypes.c_uint32), ("N", ctypes.c_int64),
                ("K", ctypes.c_int64), ("bits", ctypes.c_int32), ("block_size", ctypes.c_int32),
                ("scale_dtype", ctypes.c_int32), ("has_zp", ctypes.c_int32), ("row_stride", ctypes.c_int64),
                ("scale_offset", ctypes.c_int64), ("zp_offset", ctypes.c_int64), ("bytes", ctypes.c_int64),
                ("identity", ctypes.c_uint64)]


class KvCacheDesc(ctypes.Structure):
    """kv_cache_desc: a paged key-value cache (see kv_cache)."""
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("num_pages", ctypes.c_int64),
                ("page_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64), ("token_stride", ctypes.c_int64),
                ("page_size", ctypes.c_int32), ("kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("k_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p),
                ("scale_page_stride", ctypes.c_int64), ("scale_head_stride", ctypes.c_int64),
                ("scale_block", ctypes.c_int32)]
    device = None  # of the tensors, where kv_cache saw them


class KvStepDesc(ctypes.Structure):
    """kv_step_desc: the new tokens of one step (see kv_step)."""
    _fields_ = [("seq_lens", ctypes.c_void_p), ("new_start", ctypes.c_void_p), ("page_table", ctypes.c_void_p),
                ("table_stride", ctypes.c_int64), ("batch", ctypes.c_int32), ("tokens", ctypes.c_int32),
                ("max_new", ctypes.c_int32), ("max_pages", ctypes.c_int32)]
    device = None


class KvRopeDesc(ctypes.Structure):
    """kv_rope_desc: per-head norms and position rotation (see kv_rope)."""
    _fields_ = [("cos_sin", ctypes.c_void_p), ("max_pos", ctypes.c_int64), ("rot_dim", ctypes.c_int32),
                ("interleaved", ctypes.c_int32), ("q_norm", ctypes.c_void_p), ("k_norm", ctypes.c_void_p),
                ("eps", ctypes.c_float)]
    device = None
    norm_dim = None  # length of the norms' weights, where kv_rope saw them


class KvPoolDesc(ctypes.Structure):
    """kv_pool_desc: the pages of a pool (see kv_pool)."""
    _fields_ = [("held", ctypes.c_void_p), ("page_table", ctypes.c_void_p), ("table_stride", ctypes.c_int64),
                ("free_pages", ctypes.c_void_p), ("free_count", ctypes.c_void_p), ("held_out", ctypes.c_void_p),
                ("free_count_out", ctypes.c_void_p), ("batch", ctypes.c_int32), ("max_pages", ctypes.c_int32),
                ("num_pages", ctypes.c_int32), ("page_size", ctypes.c_int32)]
    device = None


class TokenRules(ctypes.Structure):
    """token_rules: penalties, biases and temperatures of a batch (see token_rules)."""
    _fields_ = [("temperature", ctypes.c_void_p), ("history", ctypes.c_void_p), ("history_stride", ctypes.c_int64),
                ("history_lens", ctypes.c_void_p), ("prompt_lens", ctypes.c_void_p), ("repetition", ctypes.c_void_p),
                ("frequency", ctypes.c_void_p), ("presence", ctypes.c_void_p), ("bias_tokens", ctypes.c_void_p),
                ("bias_values", ctypes.c_void_p), ("bias_stride", ctypes.c_int64), ("batch", ctypes.c_int32),
                ("history_columns", ctypes.c_int32), ("biases", ctypes.c_int32)]
    device = None


class MnbError(RuntimeError):
    def __init__(self, status: int, call: str):
        super().__init__(f"{call} failed: {STATUS.get(status, status)}")
        self.status = status
        self.call = call


_address = ctypes.addressof
_P = ctypes.c_void_p
_I64 = ctypes.c_int64
_I = ctypes.c_int
_SZ = ctypes.c_size_t

_SIGNATURES = {
    "mnb_matmul_workspace_size": [_I64, _I64, _I64, _I, _I, _I, ctypes.POINTER(_SZ)],
    "mnb_matmul": [_P, _I, _I64, _I64, _P, _P, _I, _P, _I64, _I, _I, _P, _I, _P, _SZ, _P],
    "mnb_matmul_int8a": [_P, _I, _I64, _I64, _P, _P, _I, _P, _I64, _I, _I, _P, _I, _P],
    "mnb_gate_up_swiglu": [_P, _I, _I64, _I64, _P, _P, _I, _P, _I64, _I, _I, _I, _P, _I, _P],
    "mnb_prepack_size": [_I64, _I64, _I, _I, _I, _I, ctypes.POINTER(_SZ)],
    "mnb_prepack": [_P, _P, _I, _P, _I64, _I64, _I, _I, ctypes.c_uint64, _P, _SZ, _P, _P],
    "mnb_matmul_prepacked": [_P, _I, _I64, _I64, _P, _P, _P, _I, _P],
    "qmoe_workspace_size": [_I64, _I64, _I64, _I64, _I, _I, ctypes.POINTER(_SZ)],
    "qmoe_forward": [_P, _I, _I64, _I64, _P, _I64, _I, _I, _P, _P, _P, _I, _P, _P, _P, _I, _I64, _I, _I,
                     _P, _P, _SZ, _P],
    "qmoe_forward_ex": [_P, _I, _I64, _I64, _P, _I64, _I, _I, _P, _P, _P, _I, _P, _P, _P, _I, _I64, _I, _I,
                        _P, _P, _SZ, _P, _P],
    "qmoe_forward_static": [_P, _I, _I64, _I64, _P, _I64, _I, _I, _P, _P, _P, _I, _P, _P, _P, _I, _I64, _I, _I,
                            _P, _P],
    "qmoe_route": [_P, _I64, _I64, _I, _I, _P, _P, _P],
    "qmoe_permute": [_P, _I64, _I, _I64, _P, _P, _P, _P],
    "kv_append": [_P, _P, _P, _P, _I64, _I64, _P, _I64, _P, _I64, _I, _P, _I64, _P],
    "kv_attention_workspace_size": [_I64, _I64, _I64, _I64, ctypes.POINTER(_SZ)],
    "kv_attention": [_P, _P, _P, _I64, _I64, _I, _P, _I64, _P, ctypes.c_float, _I64, _P, _SZ, _P],
    "draft_verify": [_P, _I64, _I64, _P, _I64, _I64, _P, _P, _P, _I64, _I64, _I64, _P, _P, _P],
    "kv_plan": [_P, _P, _P, _P, _P, _I64, _P, _P, _P],
    "token_probs": [_P, _I, _I64, _I64, _P, _I64, _P, _P, _P, _I64, _I64, _I64, _I64, _P, _I64, _I64, _I, _P],
    "mnb_unpack_codes": [_P, _I64, _I64, _I, _I, _P, _P],
    "mnb_pack_codes": [_P, _I64, _I64, _I, _I, _P, _P],
    "mnb_quantize_int3": [_P, _I, _I64, _I64, _I, _P, _P, _I, _P],
    "mnb_validate_host": [_P, _P, _I, _P, _I64, _I64, _I, _I],
    "mnb_get_last_device_error": [_P],
    "mnb_diag_wait_timeout": [ctypes.c_uint64, _P],
    "mnb_status_string": [_I],
}

_LIB = None


def header_functions() -> list[str]:
    """Names of the functions include/mnb.h declares."""
    text = open(HEADER).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return re.findall(r"^\s*(?:const\s+)?\w+\s*\*?\s*(\w+)\s*\(", text, flags=re.M)


def load_library(path: str | None = None):
    global _LIB
    if _LIB is None:
        p = path or os.environ.get("MNB_LIBRARY", DEFAULT_LIB)
        if not os.path.exists(p):
            raise ImportError(f"libmnb.so is not built ({p}); run __graft_entry__.build()")
        lib = ctypes.CDLL(p)
        for name, args in _SIGNATURES.items():
            fn = getattr(lib, name)
            fn.argtypes = args
            fn.restype = ctypes.c_char_p if name == "mnb_status_string" else _I
        _LIB = lib
    return _LIB


def library_path() -> str:
    return DEFAULT_LIB


# ------------------------------------------------------------- marshalling

_DTYPE_CODES = {}


def _dtype_code(t) -> int:
    code = _DTYPE_CODES.get(t.dtype)
    if code is None:
        import torch
        _DTYPE_CODES.update({torch.float32: F32, torch.float16: F16, torch.bfloat16: BF16})
        if t.dtype not in _DTYPE_CODES:
            raise TypeError(f"unsupported dtype {t.dtype}")
        code = _DTYPE_CODES[t.dtype]
    return code


def _ptr(x):
    if x is None:
        return None
    if isinstance(x, int):
        return x
    if not x.is_contiguous():
        raise ValueError("tensors passed to the library must be contiguous")
    return x.data_ptr()


def _stream(stream):
    if stream is None:
        import torch
        # the raw handle of torch.cuda.current_stream(), without building a Stream object (3 us a call)
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _stream_for(t, stream):
    """_stream for a call on the tensor t: the library launches on the current device, so t may not be on another GPU."""
    import torch
    device = torch.cuda.current_device()
    if not isinstance(t, int) and t.get_device() not in (device, -1):
        raise ValueError(f"the tensors are on CUDA device {t.get_device()}, the current device is {device}")
    return torch._C._cuda_getCurrentRawStream(device) if stream is None else _stream(stream)


def _check(status: int, call: str):
    if status != 0:
        raise MnbError(status, call)


# ------------------------------------------------------------- entry points

def mnb_status_string(status: int) -> str:
    return load_library().mnb_status_string(status).decode()


def mnb_matmul_workspace_size(M, K, N, bits, block_size, a_dtype=F32) -> int:
    out = _SZ(0)
    _check(load_library().mnb_matmul_workspace_size(M, K, N, bits, block_size, a_dtype, ctypes.byref(out)),
           "mnb_matmul_workspace_size")
    return out.value


def mnb_matmul(A, B_packed, scales, zero_points, N, bits, block_size, Y, workspace=None, stream=None,
               *, K=None, M=None, a_dtype=None, scale_dtype=None, y_dtype=None, check=True):
    """Y[M, N] = A[M, K] . dequant(B_packed, scales, zero_points)^T."""
    if K is None:
        K = A.shape[-1]
    if M is None:
        M = A.numel() // K
    a_dtype = _dtype_code(A) if a_dtype is None else a_dtype
    scale_dtype = _dtype_code(scales) if scale_dtype is None else scale_dtype
    y_dtype = _dtype_code(Y) if y_dtype is None else y_dtype
    if workspace is None:  # the workspace the library can use (split-K partial sums), if any
        need = mnb_matmul_workspace_size(M, K, N, bits, block_size, a_dtype)
        if need:
            import torch
            workspace = torch.empty(need, dtype=torch.uint8, device=A.device)
    ws_bytes = 0 if workspace is None or isinstance(workspace, int) else workspace.numel() * workspace.element_size()
    st = load_library().mnb_matmul(_ptr(A), a_dtype, M, K, _ptr(B_packed), _ptr(scales), scale_dtype,
                                   _ptr(zero_points), N, bits, block_size, _ptr(Y), y_dtype, _ptr(workspace),
                                   ws_bytes, _stream_for(A, stream))
    if check:
        _check(st, "mnb_matmul")
    return st


def mnb_matmul_int8a(A, B_packed, scales, zero_points, N, bits, block_size, Y, stream=None, *, K=None, M=None,
                     a_dtype=None, scale_dtype=None, y_dtype=None, check=True):
    """Y[M, N] = A . dequant(B)^T with A quantised per (row, block) to int8 (accuracy_level=4)."""
    if K is None:
        K = A.shape[-1]
    if M is None:
        M = A.numel() // K
    a_dtype = _dtype_code(A) if a_dtype is None else a_dtype
    scale_dtype = _dtype_code(scales) if scale_dtype is None else scale_dtype
    y_dtype = _dtype_code(Y) if y_dtype is None else y_dtype
    st = load_library().mnb_matmul_int8a(_ptr(A), a_dtype, M, K, _ptr(B_packed), _ptr(scales), scale_dtype,
                                         _ptr(zero_points), N, bits, block_size, _ptr(Y), y_dtype,
                                         _stream_for(A, stream))
    if check:
        _check(st, "mnb_matmul_int8a")
    return st


def mnb_gate_up_swiglu(A, B_packed, scales, zero_points, I, bits, block_size, Y, stream=None, *,
                       layout=FC1_INTERLEAVED, K=None, M=None, a_dtype=None, scale_dtype=None, y_dtype=None,
                       check=True):
    """Y[M, I] = silu(A . Wgate^T) * (A . Wup^T) from the fused gate/up weight [2I, K]."""
    if K is None:
        K = A.shape[-1]
    if M is None:
        M = A.numel() // K
    a_dtype = _dtype_code(A) if a_dtype is None else a_dtype
    scale_dtype = _dtype_code(scales) if scale_dtype is None else scale_dtype
    y_dtype = _dtype_code(Y) if y_dtype is None else y_dtype
    st = load_library().mnb_gate_up_swiglu(_ptr(A), a_dtype, M, K, _ptr(B_packed), _ptr(scales), scale_dtype,
                                           _ptr(zero_points), I, bits, block_size, layout, _ptr(Y), y_dtype,
                                           _stream_for(A, stream))
    if check:
        _check(st, "mnb_gate_up_swiglu")
    return st


def mnb_prepack_size(N, K, bits, block_size, scale_dtype=F32, has_zero_points=False) -> int:
    out = _SZ(0)
    _check(load_library().mnb_prepack_size(N, K, bits, block_size, scale_dtype, int(bool(has_zero_points)),
                                           ctypes.byref(out)), "mnb_prepack_size")
    return out.value


def mnb_prepack(B_packed, scales, zero_points, N, K, bits, block_size, dst, identity=0, stream=None, *,
                scale_dtype=None, dst_bytes=None, check=True):
    """Writes the version-1 prepacked form of a row-local weight into `dst`; returns its
    PrepackedDesc (with check=False: (status, desc))."""
    scale_dtype = _dtype_code(scales) if scale_dtype is None else scale_dtype
    if dst_bytes is None:
        dst_bytes = dst.numel() * dst.element_size()
    desc = PrepackedDesc()
    st = load_library().mnb_prepack(_ptr(B_packed), _ptr(scales), scale_dtype, _ptr(zero_points), N, K, bits,
                                    block_size, ctypes.c_uint64(identity), _ptr(dst), dst_bytes, ctypes.byref(desc),
                                    _stream_for(B_packed, stream))
    if not check:
        return st, desc
    _check(st, "mnb_prepack")
    return desc


def mnb_matmul_prepacked(A, desc, prepacked, Y, stream=None, *, K=None, M=None, a_dtype=None, y_dtype=None,
                         check=True):
    """Y[M, N] = A . W^T with W read from a prepacked buffer and its descriptor."""
    if K is None:
        K = A.shape[-1]
    if M is None:
        M = A.numel() // K
    a_dtype = _dtype_code(A) if a_dtype is None else a_dtype
    y_dtype = _dtype_code(Y) if y_dtype is None else y_dtype
    st = load_library().mnb_matmul_prepacked(_ptr(A), a_dtype, M, K, ctypes.byref(desc), _ptr(prepacked), _ptr(Y),
                                             y_dtype, _stream_for(A, stream))
    if check:
        _check(st, "mnb_matmul_prepacked")
    return st


def qmoe_workspace_size(T, H, I, E, k, act_dtype=F16) -> int:
    out = _SZ(0)
    _check(load_library().qmoe_workspace_size(T, H, I, E, k, act_dtype, ctypes.byref(out)),
           "qmoe_workspace_size")
    return out.value


def qmoe_forward(X, router_logits, k, normalize_topk, fc1_w, fc1_scales, fc1_zp, fc1_bits, fc2_w, fc2_scales,
                 fc2_zp, fc2_bits, I, block_size, Y, workspace, stream=None, *, fc1_layout=FC1_INTERLEAVED,
                 T=None, H=None, E=None, act_dtype=None, workspace_bytes=None, check=True):
    """One QMoE expert-FFN layer: Y[T, H] from X[T, H] and router_logits[T, E]."""
    if H is None:
        H = X.shape[-1]
    if T is None:
        T = X.numel() // H
    if E is None:
        E = router_logits.shape[-1]
    act_dtype = _dtype_code(X) if act_dtype is None else act_dtype
    if workspace_bytes is None:
        workspace_bytes = workspace.numel() * workspace.element_size()
    st = load_library().qmoe_forward(_ptr(X), act_dtype, T, H, _ptr(router_logits), E, k, int(bool(normalize_topk)),
                                     _ptr(fc1_w), _ptr(fc1_scales), _ptr(fc1_zp), fc1_bits, _ptr(fc2_w),
                                     _ptr(fc2_scales), _ptr(fc2_zp), fc2_bits, I, block_size, fc1_layout, _ptr(Y),
                                     _ptr(workspace), workspace_bytes, _stream_for(X, stream))
    if check:
        _check(st, "qmoe_forward")
    return st


class QmoeOptions(ctypes.Structure):
    """The qmoe_options struct of include/mnb.h (device pointers as ints)."""
    _fields_ = [("fc1_bias", ctypes.c_void_p), ("fc2_bias", ctypes.c_void_p), ("agg_weights", ctypes.c_void_p),
                ("agg_dtype", ctypes.c_int), ("logits_dtype", ctypes.c_int)]


def qmoe_forward_ex(X, router_logits, k, normalize_topk, fc1_w, fc1_scales, fc1_zp, fc1_bits, fc2_w, fc2_scales,
                    fc2_zp, fc2_bits, I, block_size, Y, workspace, stream=None, *, fc1_bias=None, fc2_bias=None,
                    agg_weights=None, fc1_layout=FC1_INTERLEAVED, T=None, H=None, E=None, act_dtype=None,
                    workspace_bytes=None, check=True):
    """qmoe_forward with the optional inputs: FC1/FC2 biases, aggregation weights
    [T, E], router logits of any float dtype (taken from the tensor)."""
    if H is None:
        H = X.shape[-1]
    if T is None:
        T = X.numel() // H
    if E is None:
        E = router_logits.shape[-1]
    act_dtype = _dtype_code(X) if act_dtype is None else act_dtype
    if workspace_bytes is None:
        workspace_bytes = workspace.numel() * workspace.element_size()
    opts = QmoeOptions(_ptr(fc1_bias), _ptr(fc2_bias), _ptr(agg_weights),
                       _dtype_code(agg_weights) if agg_weights is not None else F32, _dtype_code(router_logits))
    st = load_library().qmoe_forward_ex(_ptr(X), act_dtype, T, H, _ptr(router_logits), E, k, int(bool(normalize_topk)),
                                        _ptr(fc1_w), _ptr(fc1_scales), _ptr(fc1_zp), fc1_bits, _ptr(fc2_w),
                                        _ptr(fc2_scales), _ptr(fc2_zp), fc2_bits, I, block_size, fc1_layout, _ptr(Y),
                                        _ptr(workspace), workspace_bytes, ctypes.byref(opts), _stream_for(X, stream))
    if check:
        _check(st, "qmoe_forward_ex")
    return st


def qmoe_forward_static(X, router_logits, k, normalize_topk, fc1_w, fc1_scales, fc1_zp, fc1_bits, fc2_w,
                        fc2_scales, fc2_zp, fc2_bits, I, block_size, Y, stream=None, *, fc1_layout=FC1_INTERLEAVED,
                        T=None, H=None, E=None, act_dtype=None, check=True):
    """qmoe_forward with the library's fixed 8 MiB scratch instead of a caller workspace."""
    if H is None:
        H = X.shape[-1]
    if T is None:
        T = X.numel() // H
    if E is None:
        E = router_logits.shape[-1]
    act_dtype = _dtype_code(X) if act_dtype is None else act_dtype
    st = load_library().qmoe_forward_static(_ptr(X), act_dtype, T, H, _ptr(router_logits), E, k,
                                            int(bool(normalize_topk)), _ptr(fc1_w), _ptr(fc1_scales), _ptr(fc1_zp),
                                            fc1_bits, _ptr(fc2_w), _ptr(fc2_scales), _ptr(fc2_zp), fc2_bits, I,
                                            block_size, fc1_layout, _ptr(Y), _stream_for(X, stream))
    if check:
        _check(st, "qmoe_forward_static")
    return st


def qmoe_route(logits, k, normalize_topk, topk_idx, topk_w, stream=None, *, T=None, E=None, check=True):
    if E is None:
        E = logits.shape[-1]
    if T is None:
        T = logits.numel() // E
    st = load_library().qmoe_route(_ptr(logits), T, E, k, int(bool(normalize_topk)), _ptr(topk_idx), _ptr(topk_w),
                                   _stream_for(logits, stream))
    if check:
        _check(st, "qmoe_route")
    return st


def qmoe_permute(topk_idx, E, counts, offsets, perm, stream=None, *, T=None, k=None, check=True):
    if k is None:
        k = topk_idx.shape[-1]
    if T is None:
        T = topk_idx.numel() // k
    st = load_library().qmoe_permute(_ptr(topk_idx), T, k, E, _ptr(counts), _ptr(offsets), _ptr(perm),
                                     _stream_for(topk_idx, stream))
    if check:
        _check(st, "qmoe_permute")
    return st


def _device_of(t, name) -> int:
    """The device of a CUDA tensor."""
    if t.get_device() < 0:
        raise ValueError(f"{name} must be a CUDA tensor")
    return t.get_device()


def _elsewhere(t, name, device):
    return ValueError(f"{name} must be a CUDA tensor" if t.get_device() < 0 else
                      f"{name} must be on CUDA device {device} like the other tensors, not on {t.get_device()}")


def _on_gpu(t, name, dtype, device):
    """The data pointer of a tensor on `device` (None stays None)."""
    if t is None:
        return None
    if t.get_device() != device:
        raise _elsewhere(t, name, device)
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, not {t.dtype}")
    return t.data_ptr()


def _packed(t, name, dtype, device, shape=None):
    """_on_gpu of a contiguous tensor, of `shape` where that is given."""
    if t is None:
        return None
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if t.get_device() != device:
        raise _elsewhere(t, name, device)
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, not {t.dtype}")
    return t.data_ptr()


def _described(device, *descriptors):
    """Refuses descriptors of tensors that are not on `device` (None: the caller built the descriptor)."""
    for d in descriptors:
        if d.device != device and d.device is not None:
            raise ValueError(f"{type(d).__name__} of tensors on CUDA device {d.device}, not on {device} like the others")


def kv_cache(k, v, k_scale=None, v_scale=None) -> KvCacheDesc:
    """Describes a paged cache held in k and v [pages, kv_heads, page_size, head_dim] (f16 or bf16; any strides
    with unit stride along head_dim, the same for both: permuted views describe other layouts).  A cache of 8-bit codes
    has k and v in float8_e4m3fn and k_scale, v_scale f32 [pages, kv_heads, page_size / block]: element = code * scale
    (any strides with unit stride along the blocks, the same for both)."""
    import torch
    if k.shape != v.shape or k.stride() != v.stride() or k.dtype != v.dtype or k.dim() != 4:
        raise ValueError("k and v must be 4-D tensors of one shape, dtype and layout")
    if k.stride(3) != 1:
        raise ValueError("the head dimension must have unit stride")
    device = _device_of(k, "k")
    codes = k.dtype == torch.float8_e4m3fn
    if codes != (k_scale is not None) or codes != (v_scale is not None):
        raise ValueError("a cache of float8_e4m3fn has k_scale and v_scale, others have none")
    d = KvCacheDesc(_on_gpu(k, "k", None, device), _on_gpu(v, "v", None, device), k.shape[0], k.stride(0), k.stride(1),
                    k.stride(2), k.shape[2], k.shape[1], k.shape[3], E4M3 if codes else _dtype_code(k))
    if codes:
        blocks = k_scale.shape[2] if k_scale.dim() == 3 else 0
        if k_scale.shape != v_scale.shape or k_scale.stride() != v_scale.stride() or blocks < 1 or \
                k_scale.shape != (k.shape[0], k.shape[1], blocks) or k.shape[2] % blocks:
            raise ValueError("k_scale and v_scale must be [pages, kv_heads, page_size / block], of one layout")
        if blocks > 1 and k_scale.stride(2) != 1:
            raise ValueError("the scales must have unit stride along the blocks")
        d.k_scale, d.v_scale = _on_gpu(k_scale, "k_scale", torch.float32, device), _on_gpu(v_scale, "v_scale", torch.float32, device)
        d.scale_page_stride, d.scale_head_stride = k_scale.stride(0), k_scale.stride(1)
        d.scale_block = k.shape[2] // blocks
    d.tensors, d.device = (k, v, k_scale, v_scale), device  # (the tensors live as long as the descriptor)
    return d


def kv_step(seq_lens, page_table, new_start=None, tokens=None, max_new=1) -> KvStepDesc:
    """Describes a step's new tokens: seq_lens int32 [batch] (with the new tokens), page_table int32 [batch,
    max_pages] (unit stride along pages), new_start int32 [batch + 1] or None for one token per sequence (then
    `tokens` is the batch).  max_new: the most new tokens of one sequence."""
    import torch
    batch = seq_lens.shape[0]
    if tokens is None:
        if new_start is not None:
            raise ValueError("tokens must be given with new_start")
        tokens = batch
    if page_table.dim() != 2 or page_table.shape[0] != batch or (page_table.shape[1] > 1 and page_table.stride(1) != 1):
        raise ValueError("page_table must be [batch, max_pages] with unit stride along the pages")
    if new_start is not None and new_start.numel() != batch + 1:
        raise ValueError("new_start must have batch + 1 elements")
    stride = page_table.stride(0) if batch > 1 else max(page_table.shape[1], 1)
    device = _device_of(seq_lens, "seq_lens")
    d = KvStepDesc(_packed(seq_lens, "seq_lens", torch.int32, device), _packed(new_start, "new_start", torch.int32, device),
                   _on_gpu(page_table, "page_table", torch.int32, device), stride, batch, tokens, max_new,
                   page_table.shape[1])
    d.tensors, d.device = (seq_lens, new_start, page_table), device
    return d


def kv_pool(held, page_table, free_pages, free_count, page_size, *, held_out=None, free_count_out=None) -> KvPoolDesc:
    """Describes a pool of pages: held int32 [batch], page_table int32 [batch, max_pages] (unit stride along pages),
    free_pages int32 [num_pages] (a stack, the last free page on top), free_count int32 [1].  held_out and
    free_count_out get the state after a step (None: held and free_count themselves)."""
    import torch
    i32, batch = torch.int32, held.shape[0]
    device = _device_of(held, "held")
    if page_table.dim() != 2 or page_table.shape[0] != batch or (page_table.shape[1] > 1 and page_table.stride(1) != 1):
        raise ValueError("page_table must be [batch, max_pages] with unit stride along the pages")
    if free_pages.dim() != 1:
        raise ValueError("free_pages must be [num_pages]")
    held_out = held if held_out is None else held_out
    free_count_out = free_count if free_count_out is None else free_count_out
    columns = page_table.shape[1]
    d = KvPoolDesc(_packed(held, "held", i32, device, (batch,)), _on_gpu(page_table, "page_table", i32, device),
                   page_table.stride(0) if batch > 1 else max(columns, 1), _packed(free_pages, "free_pages", i32, device),
                   _packed(free_count, "free_count", i32, device, (1,)), _packed(held_out, "held_out", i32, device, (batch,)),
                   _packed(free_count_out, "free_count_out", i32, device, (1,)), batch, columns, free_pages.shape[0],
                   page_size)
    d.tensors, d.device = (held, page_table, free_pages, free_count, held_out, free_count_out), device
    return d


def kv_plan(pool, keep, new, seq_lens, new_start, *, slots=None, max_tokens=None, refused=None, stream=None, check=True):
    """Plans a step: each sequence keeps its first keep int32 [batch] tokens and gets new int32 [batch] more.  Writes
    seq_lens int32 [batch] and new_start int32 [batch + 1] for kv_step, page tables and free pages in the pool, slots
    int64 [max_tokens] (page * page_size + row of each new token) and refused int32 [batch].  max_tokens: the most new
    tokens of the step (default: the slots' length, without slots 2^30)."""
    import torch
    i32, shape, device = torch.int32, (pool.batch,), keep.get_device()
    if pool.device != device:
        _described(device, pool)
    sp = None
    if slots is not None:
        sp = _packed(slots, "slots", torch.int64, device)
        if max_tokens is None:
            max_tokens = slots.numel()
        elif max_tokens > slots.numel():
            raise ValueError("slots must have max_tokens elements")
    elif max_tokens is None:
        max_tokens = 1 << 30
    st = load_library().kv_plan(_address(pool), _packed(keep, "keep", i32, device, shape),
                                _packed(new, "new", i32, device, shape), _packed(seq_lens, "seq_lens", i32, device, shape),
                                _packed(new_start, "new_start", i32, device, (pool.batch + 1,)), max_tokens, sp,
                                _packed(refused, "refused", i32, device, shape), _stream_on(device, stream))
    if check:
        _check(st, "kv_plan")
    return st


def kv_rope(cos_sin=None, *, interleaved=False, q_norm=None, k_norm=None, eps=1e-6) -> KvRopeDesc:
    """Describes the rotation (cos_sin f32 [max_pos, rot_dim]: cosines, then sines) and the per-head norms (f32
    [head_dim]) of queries and keys; None leaves a part out."""
    import torch
    max_pos, rot_dim = (0, 0) if cos_sin is None else cos_sin.shape
    lengths = {w.numel() for w in (q_norm, k_norm) if w is not None}
    if len(lengths) > 1:
        raise ValueError("q_norm and k_norm must have one length")
    device = next((_device_of(t, "a tensor of the rope") for t in (cos_sin, q_norm, k_norm) if t is not None), None)
    d = KvRopeDesc(_packed(cos_sin, "cos_sin", torch.float32, device), max_pos, rot_dim, int(bool(interleaved)),
                   _packed(q_norm, "q_norm", torch.float32, device), _packed(k_norm, "k_norm", torch.float32, device), eps)
    d.tensors, d.device = (cos_sin, q_norm, k_norm), device
    if lengths:
        d.norm_dim = lengths.pop()
    return d


def _token_rows(t, name, shape, device):
    """Pointer and token stride of rows [tokens, heads, head_dim] (heads adjacent within a token)."""
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, not {list(t.shape)}")
    stride = t.stride()
    if stride[2] != 1 or (stride[1] != shape[2] and shape[1] > 1):
        raise ValueError(f"the heads of a token of {name} must be adjacent")
    if t.get_device() != device:
        raise _elsewhere(t, name, device)
    return t.data_ptr(), (stride[0] if shape[0] > 1 else shape[1] * shape[2])  # one token's stride is never used


_torch_c = None  # torch's C module, once a call has imported torch


def _stream_on(device, stream):
    """The raw handle of `stream`, or of the current stream.  The library launches on the current device: `device`, where
    the tensors are, has to be that one."""
    global _torch_c
    if _torch_c is None:
        import torch
        _torch_c = torch._C
    if device < 0 or device != _torch_c._cuda_getDevice():
        raise ValueError("the tensors must be on the current CUDA device, not on " +
                         ("the host" if device < 0 else f"CUDA device {device}"))
    return _torch_c._cuda_getCurrentRawStream(device) if stream is None else _stream(stream)


def kv_append(cache, step, q, k, v, q_out, rope=None, stream=None, *, check=True):
    """Stores a step's k and v [tokens, kv_heads, head_dim] in the cache and writes q [tokens, q_heads, head_dim] to
    q_out (may be q; both None: no queries), q and k normed and rotated as `rope` says.  Rows may be strided parts
    of one projection's output."""
    n, dim, dtype, device = step.tokens, cache.head_dim, k.dtype, k.get_device()
    if not cache.device == step.device == device:
        _described(device, cache, step)
    shape = (n, cache.kv_heads, dim)
    kp, ks = _token_rows(k, "k", shape, device)
    vp, vs = _token_rows(v, "v", shape, device)
    qp = op = None
    qs = os_ = heads = 0
    if q is not None:
        shape = q.shape
        heads = shape[1]
        qp, qs = _token_rows(q, "q", (n, heads, dim), device)
        if q_out is not None:
            op, os_ = _token_rows(q_out, "q_out", shape, device)
            if q_out.dtype != dtype:
                raise TypeError("q_out must have q's dtype")
        if q.dtype != dtype:
            raise TypeError("q, k and v must have one dtype")
    elif q_out is not None:
        raise ValueError("q_out needs q")
    if v.dtype != dtype:
        raise TypeError("q, k and v must have one dtype")
    if rope is not None:
        if rope.device != device:
            _described(device, rope)
        if rope.norm_dim != dim and rope.norm_dim is not None:
            raise ValueError(f"q_norm and k_norm must have head_dim = {dim} elements, not {rope.norm_dim}")
    st = load_library().kv_append(_address(cache), _address(step), None if rope is None else _address(rope), qp, qs, heads,
                                  kp, ks, vp, vs, _dtype_code(k), op, os_, _stream_on(device, stream))
    if check:
        _check(st, "kv_append")
    return st


def kv_attention_workspace_size(q_heads, kv_heads, head_dim, max_new=1) -> int:
    out = _SZ(0)
    _check(load_library().kv_attention_workspace_size(q_heads, kv_heads, head_dim, max_new, ctypes.byref(out)),
           "kv_attention_workspace_size")
    return out.value


def kv_attention(cache, step, q, out, workspace=None, *, scale=None, window=0, lse=None, stream=None, check=True):
    """Attention of the step's new tokens q [tokens, q_heads, head_dim] over the cache into out (same shape and
    dtype); scale defaults to head_dim ** -0.5, lse (f32 [tokens, q_heads]) is optional."""
    n, dim, shape, device = step.tokens, cache.head_dim, q.shape, q.get_device()
    if not cache.device == step.device == device:
        _described(device, cache, step)
    heads = shape[1]
    qp, qs = _token_rows(q, "q", (n, heads, dim), device)
    op, os_ = _token_rows(out, "out", shape, device)
    if out.dtype != q.dtype:
        raise TypeError("out must have q's dtype")
    lp = None
    if lse is not None:
        import torch
        lp = _packed(lse, "lse", torch.float32, device)
        if lse.numel() != n * heads:
            raise ValueError("lse must be [tokens, q_heads]")
    if workspace is None:
        import torch
        workspace = torch.empty(kv_attention_workspace_size(heads, cache.kv_heads, dim, step.max_new),
                                dtype=torch.uint8, device=q.device)
        if stream is not None:  # the allocation belongs to the current stream and is given back at return
            workspace.record_stream(stream if not isinstance(stream, int) else torch.cuda.ExternalStream(stream))
    st = load_library().kv_attention(_address(cache), _address(step), qp, qs, heads, _dtype_code(q), op, os_,
                                     lp, dim ** -0.5 if scale is None else scale, window,
                                     _packed(workspace, "workspace", None, device), workspace.nbytes,
                                     _stream_on(device, stream))
    if check:
        _check(st, "kv_attention")
    return st


def token_rules(*, batch=None, temperature=None, history=None, history_lens=None, prompt_lens=None, repetition=None,
                frequency=None, presence=None, bias_tokens=None, bias_values=None) -> TokenRules:
    """Describes what changes a batch's logits: temperature, repetition, frequency, presence f32 [batch]; history int32
    [batch, columns] (unit stride along the tokens) with history_lens and prompt_lens int32 [batch]; bias_tokens int32
    and bias_values f32 [batch, biases] of one layout.  None leaves a part out; `batch` is needed where all are None."""
    import torch
    given = [t for t in (temperature, history, history_lens, prompt_lens, repetition, frequency, presence, bias_tokens,
                         bias_values) if t is not None]
    device = _device_of(given[0], "a tensor of the rules") if given else None
    if batch is None:
        if not given:
            raise ValueError("batch must be given where there are no rules")
        batch = given[0].shape[0]
    if (history is None) != (history_lens is None) or (history is None and prompt_lens is not None):
        raise ValueError("history and history_lens belong together, prompt_lens needs them")
    if (bias_tokens is None) != (bias_values is None):
        raise ValueError("bias_tokens and bias_values belong together")
    f32, i32 = torch.float32, torch.int32

    def numbers(t, name, dtype=f32):
        return _packed(t, name, dtype, device, (batch,))

    def rows(t, name, dtype):
        if t is None:
            return None, 0, 0
        if t.dim() != 2 or t.shape[0] != batch or (t.shape[1] > 1 and t.stride(1) != 1):
            raise ValueError(f"{name} must be [batch, any] with unit stride along a row")
        return _on_gpu(t, name, dtype, device), (t.stride(0) if batch > 1 else t.shape[1]), t.shape[1]

    hp, hs, columns = rows(history, "history", i32)
    tp, ts, biases = rows(bias_tokens, "bias_tokens", i32)
    vp, vs, values = rows(bias_values, "bias_values", f32)
    if (ts, biases) != (vs, values):
        raise ValueError("bias_tokens and bias_values must have one shape and layout")
    if columns == 0:
        hp = None
    d = TokenRules(numbers(temperature, "temperature"), hp, hs, numbers(history_lens, "history_lens", i32),
                   numbers(prompt_lens, "prompt_lens", i32), numbers(repetition, "repetition"),
                   numbers(frequency, "frequency"), numbers(presence, "presence"), tp, vp, ts, batch, columns, biases)
    d.tensors = (temperature, history, history_lens, prompt_lens, repetition, frequency, presence, bias_tokens, bias_values)
    d.device = device
    return d


def token_probs(logits, rules, out, *, row_start=None, draft_tokens=None, mask=None, softmax=True, stream=None, check=True):
    """Writes to out f32 [batch, rows, vocab] the probabilities of a step's logits (softmax=False: the changed logits)
    under `rules`: logits f32, f16 or bf16 [batch, rows, vocab], or [tokens, vocab] with row_start int32 [batch + 1]
    (row i of sequence b is row_start[b] + i).  draft_tokens int32 [batch, rows - 1]: row i follows the first i of
    them.  mask int32 [batch, rows, ceil(vocab / 32)]: bits of the allowed tokens.  Unit stride along the vocabulary;
    out may be fp32 logits."""
    import torch
    batch, rows, vocab = out.shape
    device = out.get_device()
    if rules.batch != batch:
        raise ValueError(f"out must have the rules' batch of {rules.batch} sequences")
    if rules.device != device and rules.device is not None:
        _described(device, rules)

    def rows_of(t, name, dtype, width):  # pointer and strides (those of an extent of one are never used)
        s0, s1, s2 = t.stride()
        if s2 != 1 and width > 1:
            raise ValueError(f"{name} must have unit stride along its rows")
        return _on_gpu(t, name, dtype, device), (s0 if batch > 1 else rows * width), (s1 if rows > 1 else width)

    tokens = 0
    if row_start is None:
        if logits.shape != out.shape:
            raise ValueError(f"logits must be {list(out.shape)}, or [tokens, vocab] with row_start")
        lp, ls, lr = rows_of(logits, "logits", None, vocab)
    else:
        if logits.dim() != 2 or logits.shape[1] != vocab or (vocab > 1 and logits.stride(1) != 1):
            raise ValueError("logits must be [tokens, vocab] with unit stride along the vocabulary")
        tokens = logits.shape[0]
        lp, ls, lr = _on_gpu(logits, "logits", None, device), 0, (logits.stride(0) if tokens > 1 else vocab)
    op, os_, orow = rows_of(out, "out", torch.float32, vocab)
    mp, ms, mr = None, 0, 0
    if mask is not None:
        words = (vocab + 31) // 32
        if mask.shape != (batch, rows, words):
            raise ValueError(f"mask must be {[batch, rows, words]}")
        mp, ms, mr = rows_of(mask, "mask", torch.int32, words)
    st = load_library().token_probs(lp, _dtype_code(logits), ls, lr,
                                    _packed(row_start, "row_start", torch.int32, device, (batch + 1,)), tokens,
                                    _address(rules),
                                    _packed(draft_tokens, "draft_tokens", torch.int32, device, (batch, max(rows - 1, 0))), mp, ms,
                                    mr, rows, vocab, op, os_, orow, int(bool(softmax)), _stream_on(device, stream))
    if check:
        _check(st, "token_probs")
    return st


def draft_verify(target, draft, draft_tokens, uniforms, tokens, accepted, *, n_drafts=None, stream=None, check=True):
    """Verifies draft_tokens int32 [batch, n] against target f32 [batch, n + 1, vocab] (draft f32 [batch, n, vocab], or
    None for drafts without probabilities) with uniforms f32 [batch, n + 1]; writes tokens int32 [batch, n + 1]
    (standing drafts, the drawn token, -1s) and accepted int32 [batch]."""
    import torch
    batch, rows, vocab = target.shape
    n, f32, i32, device = rows - 1, torch.float32, torch.int32, target.get_device()
    if draft is not None and draft.shape != (batch, n, vocab):
        raise ValueError("draft must be [batch, n, vocab]")
    if n == 0:
        draft = None  # nothing was drafted

    def rows_of(t, name, count):  # pointer and strides (those of an extent of one are never used)
        s0, s1, s2 = t.stride()
        if s2 != 1 and vocab > 1:
            raise ValueError(f"{name} must have unit stride along the vocabulary")
        return _on_gpu(t, name, f32, device), (s0 if batch > 1 else count * vocab), (s1 if count > 1 else vocab)

    tp, ts, tr = rows_of(target, "target", rows)
    dp, ds, dr = (None, 0, 0) if draft is None else rows_of(draft, "draft", n)
    out = (batch, rows)
    st = load_library().draft_verify(tp, ts, tr, dp, ds, dr,
                                     _packed(draft_tokens, "draft_tokens", i32, device, (batch, n)),
                                     _packed(n_drafts, "n_drafts", i32, device, (batch,)),
                                     _packed(uniforms, "uniforms", f32, device, out), batch, n, vocab,
                                     _packed(tokens, "tokens", i32, device, out),
                                     _packed(accepted, "accepted", i32, device, (batch,)), _stream_on(device, stream))
    if check:
        _check(st, "draft_verify")
    return st


def mnb_unpack_codes(B_packed, rows, K, bits, block_size, codes, stream=None, *, check=True):
    st = load_library().mnb_unpack_codes(_ptr(B_packed), rows, K, bits, block_size, _ptr(codes),
                                         _stream_for(B_packed, stream))
    if check:
        _check(st, "mnb_unpack_codes")
    return st


def mnb_pack_codes(codes, rows, K, bits, block_size, B_packed, stream=None, *, check=True):
    st = load_library().mnb_pack_codes(_ptr(codes), rows, K, bits, block_size, _ptr(B_packed), _stream_for(codes, stream))
    if check:
        _check(st, "mnb_pack_codes")
    return st


def mnb_quantize_int3(W, block_size, scale_dtype, B_packed=None, scales=None, stream=None, *, check=True):
    """INT3 quantisation of the 2-D tensor W [N, K] (f32/f16/bf16); returns
    (B_packed uint8 [N, K/bs, 3*bs/8], scales [N, K/bs] in scale_dtype), allocating
    the outputs with torch when they are not given."""
    import torch
    N, K = W.shape
    nb = K // block_size
    sdt = {F32: torch.float32, F16: torch.float16, BF16: torch.bfloat16}[scale_dtype]
    if B_packed is None:
        B_packed = torch.empty((N, nb, 3 * block_size // 8), dtype=torch.uint8, device=W.device)
    if scales is None:
        scales = torch.empty((N, nb), dtype=sdt, device=W.device)
    st = load_library().mnb_quantize_int3(_ptr(W), _dtype_code(W), N, K, block_size, _ptr(B_packed), _ptr(scales),
                                          scale_dtype, _stream_for(W, stream))
    if check:
        _check(st, "mnb_quantize_int3")
    return B_packed, scales


def mnb_validate_host(B_packed, scales, scale_dtype, zero_points, N, K, bits, block_size) -> int:
    """Host buffers (numpy arrays or ctypes-compatible objects); returns the status code."""
    def hp(a):
        if a is None:
            return None
        return a.ctypes.data_as(ctypes.c_void_p)
    return load_library().mnb_validate_host(hp(B_packed), hp(scales), scale_dtype, hp(zero_points), N, K, bits,
                                            block_size)


def mnb_get_last_device_error(stream=None) -> int:
    return load_library().mnb_get_last_device_error(_stream(stream))


def mnb_diag_wait_timeout(limit_ns: int, stream=None, *, check=True) -> int:
    """Enqueue the diagnostic kernel whose bounded wait runs out after limit_ns."""
    st = load_library().mnb_diag_wait_timeout(int(limit_ns), _stream(stream))
    if check:
        _check(st, "mnb_diag_wait_timeout")
    return st
