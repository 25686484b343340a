"""ctypes binding of libdqmoe.so: argument marshalling only.

Every function takes torch CUDA tensors, passes their data pointers, sizes and
the current CUDA stream to the C ABI of include/dqmoe.h, and raises on a
non-zero status.  No computation happens here, and there is no fallback: if
the shared library is missing the import fails.
"""
import ctypes
import os

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libdqmoe.so")

Q4_K, Q6_K, Q8_0 = 1, 2, 3
Q4_0 = 4
F32, F16, BF16 = 0, 1, 2

_P = ctypes.c_void_p
_I = ctypes.c_int
_I64 = ctypes.c_int64
_SZ = ctypes.c_size_t


class DqError(RuntimeError):
    def __init__(self, fn, status):
        self.status = status
        super().__init__("%s failed: %s (%d)" % (fn, status_string(status), status))


class MoeDesc(ctypes.Structure):
    _fields_ = [("E", ctypes.c_int32), ("top_k", ctypes.c_int32), ("hidden", ctypes.c_int32),
                ("ffn", ctypes.c_int32), ("n_shared", ctypes.c_int32), ("fmt", ctypes.c_int32),
                ("router_W", _P), ("w_gate", _P), ("w_up", _P), ("w_down", _P),
                ("sh_gate", _P), ("sh_up", _P), ("sh_down", _P)]


class MoeRoutingDesc(ctypes.Structure):
    _fields_ = [("scores", ctypes.c_int32), ("n_groups", ctypes.c_int32), ("top_groups", ctypes.c_int32),
                ("group_score", ctypes.c_int32), ("renormalize", ctypes.c_int32), ("scale", ctypes.c_float),
                ("bias", _P)]


class KvCacheDesc(ctypes.Structure):
    _fields_ = [("fmt", ctypes.c_int32), ("n_kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("n_pages", ctypes.c_int32), ("pages", _P)]


class KvRope(ctypes.Structure):
    _fields_ = [("q", _P), ("q_stride", ctypes.c_int64), ("k", _P), ("k_stride", ctypes.c_int64), ("v", _P),
                ("v_stride", ctypes.c_int64), ("dtype", ctypes.c_int32), ("n_q_heads", ctypes.c_int32),
                ("T", ctypes.c_int32), ("slots", _P), ("positions", _P), ("inv_freq", _P),
                ("rotary_dim", ctypes.c_int32), ("interleaved", ctypes.c_int32), ("factor", ctypes.c_float),
                ("q_out", _P), ("out_stride", ctypes.c_int64), ("out_dtype", ctypes.c_int32)]


class KvAttn(ctypes.Structure):
    _fields_ = [("q", _P), ("q_stride", ctypes.c_int64), ("q_dtype", ctypes.c_int32),
                ("n_q_heads", ctypes.c_int32), ("T", ctypes.c_int32), ("B", ctypes.c_int32),
                ("q_start", _P), ("kv_len", _P), ("block_table", _P),
                ("max_pages", ctypes.c_int32), ("max_q_len", ctypes.c_int32),
                ("scale", ctypes.c_float), ("causal", ctypes.c_int32), ("window", ctypes.c_int32),
                ("out", _P), ("out_stride", ctypes.c_int64), ("out_dtype", ctypes.c_int32),
                ("lse", _P)]


class KvScores(ctypes.Structure):
    _fields_ = [("softcap", ctypes.c_float), ("slopes", _P), ("prefix_len", _P), ("first_pos", _P)]


_SIGS = {
    "dq_block_geometry": [_I, _P, _P],
    "dq_dequant": [_I, _P, _I64, _P, _P],
    "dq_qgemv": [_I, _P, _I64, _I64, _P, _I, _I, _P, _P],
    "dq_qgemv_ksplit": [_I, _P, _I64, _I64, _P, _I, _I, _P, _I, _P],
    "dq_qgemv_ex": [_I, _P, _I64, _I64, _P, _I, _I, _P, _I, ctypes.c_uint, _P],
    "dq_device_status": [_P],
    "dq_stage": [_P, _P, _I64, _P],
    "dq_kv_cache_size": [_P, _P],
    "dq_kv_plan": [_P, _P, _I, _I, _P, _I, _P, _I, _P, _I, _P, _P, _P, _P, _P, _P, _P],
    "dq_kv_append": [_P, _P, _I64, _P, _I64, _I, _P, _I, _P],
    "dq_kv_append_rope": [_P, _P, _P],
    "dq_kv_read": [_P, _P, _I, _P, _P, _I, _P],
    "dq_kv_attention_workspace_size": [_P, _I, _I, _I, _I, _P],
    "dq_kv_attention": [_P, _P, _P, _SZ, _P],
    "dq_kv_attention_ex": [_P, _P, _P, _P, _SZ, _P],
}
_OPTIONAL_SIGS = {
    "dq_moe_workspace_size": [ctypes.POINTER(MoeDesc), _I, _P],
    "dq_moe_router": [_P, _I, _I, _P, _I, _I, _I, _P, _P, _P, _P],
    "dq_moe_route": [_P, _I, _I64, _I, _I, _I, _P, _P, _P, _P],
    "dq_moe_router_ex": [_P, _I, _I, _P, _I, _I, _I, _P, _P, _P, _P, _P],
    "dq_moe_forward_ex": [ctypes.POINTER(MoeDesc), _P, _P, _I, _I, _P, _P, _SZ, _P, _P, _P, _P],
    "dq_moe_forward_noalloc_ex": [ctypes.POINTER(MoeDesc), _P, _P, _I, _I, _P, _P, _P, _P, _P],
    "dq_expert_cache_set_routing": [_P, _P],
    "dq_moe_permute": [_P, _I, _I, _I, _P, _P, _P],
    "dq_moe_forward": [ctypes.POINTER(MoeDesc), _P, _I, _I, _P, _P, _SZ, _P, _P, _P, _P],
    "dq_moe_forward_noalloc": [ctypes.POINTER(MoeDesc), _P, _I, _I, _P, _P, _P, _P, _P],
    "dq_expert_cache_create": [ctypes.POINTER(MoeDesc), _I, _P, _P, _P, _I, _I, _P],
    "dq_expert_cache_workspace_size": [_P, _I, _P],
    "dq_moe_forward_streamed": [_P, _P, _I, _I, _P, _P, _SZ, _P, _P],
    "dq_expert_cache_stats": [_P, _P, _P, _P],
    "dq_expert_cache_destroy": [_P],
}


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError("libdqmoe.so is not built (run __graft_entry__.build() or "
                          "python dequant_gemv_moe_gb300/build.py)")
    lib = ctypes.CDLL(LIB_PATH)
    for name, argt in _SIGS.items():
        fn = getattr(lib, name)
        fn.argtypes = argt
        fn.restype = _I
    for name, argt in _OPTIONAL_SIGS.items():
        fn = getattr(lib, name, None)
        if fn is not None:
            fn.argtypes = argt
            fn.restype = _I
    lib.dq_status_string.argtypes = [_I]
    lib.dq_status_string.restype = ctypes.c_char_p
    return lib


lib = _load()


def status_string(status):
    return lib.dq_status_string(int(status)).decode()


def exported_symbols():
    return sorted(list(_SIGS) + list(_OPTIONAL_SIGS) + ["dq_status_string"])
