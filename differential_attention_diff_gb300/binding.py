"""ctypes binding of libdiffattn.so (the C ABI in include/diffattn.h).

Argument marshalling only: each function takes torch CUDA tensors, fills the
C parameter struct with their device pointers, sizes and element strides,
calls the entry point of the same name on the current torch stream and
raises ``DiffAttnError`` on a non-OK status.  Output and workspace buffers
that the caller does not pass are allocated here with torch (device-memory
plumbing); every computation runs in the library's kernels.  There is no
fallback: if the shared library is missing or cannot be loaded, every call
raises.
"""

from __future__ import annotations

import ctypes as C
import functools
import os
import struct
import threading

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libdiffattn.so")

DA_OK, DA_ERR_INVALID_ARG, DA_ERR_UNSUPPORTED, DA_ERR_CUDA, DA_ERR_TIMEOUT, DA_ERR_BOUNDS, \
    DA_ERR_WORKSPACE = range(7)
DA_F32, DA_BF16 = 0, 1

# Every symbol the header declares (checked by the ABI tests).
EXPORTS = (
    "diffattn_lambda_init",
    "diffattn_v1_fwd",
    "diffattn_v1_fwd_workspace_size",
    "diffattn_v1_bwd",
    "diffattn_v1_bwd_workspace_size",
    "diffattn_v1_decode",
    "diffattn_v1_decode_num_splits",
    "diffattn_v1_decode_workspace_size",
    "diffattn_v2_bwd",
    "diffattn_v2_bwd_workspace_size",
    "diffattn_grouped_fwd",
    "diffattn_grouped_fwd_workspace_size",
    "diffattn_grouped_bwd",
    "diffattn_grouped_bwd_workspace_size",
    "diffattn_v2_gate",
    "diffattn_v2_fwd",
    "diffattn_v2_fwd_workspace_size",
    "diffattn_v2_decode",
    "diffattn_v2_decode_noalloc",
    "diffattn_v2_decode_num_splits",
    "diffattn_v2_decode_workspace_size",
    "diffattn_kv4_record_bytes",
    "diffattn_kv4_append",
    "diffattn_kv4_read",
    "diffattn_v2_decode_kv4",
    "diffattn_v2_decode_kv4_workspace_size",
    "diffattn_v2_decode_weighted",
    "diffattn_v2_decode_weighted_workspace_size",
    "diffattn_kv_evict",
    "diffattn_kv_evict_workspace_size",
    "diffattn_rope_inv_freq",
    "diffattn_qk_rope_fwd",
    "diffattn_qk_rope_bwd",
    "diffattn_qk_rope_bwd_workspace_size",
    "diffattn_paged_append",
    "diffattn_v2_paged_fwd",
    "diffattn_v2_paged_fwd_workspace_size",
    "diffattn_get_device_status",
    "diffattn_debug_inject_fault",
    "diffattn_get_device_status_detail",
    "diffattn_status_string",
)


class DiffAttnError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {_status_str(status)} (status {status})")


class da_t4(C.Structure):
    _fields_ = [("ptr", C.c_void_p), ("sb", C.c_int64), ("sn", C.c_int64), ("sh", C.c_int64)]


_fp = C.POINTER(C.c_float)


class da_v1_fwd_params(C.Structure):
    _fields_ = [("B", C.c_int), ("N", C.c_int), ("H", C.c_int), ("d_qk", C.c_int), ("d_v", C.c_int),
                ("dtype", C.c_int), ("causal", C.c_int), ("softmax_scale", C.c_float),
                ("lambda_init", C.c_float), ("rms_eps", C.c_float),
                ("q1", da_t4), ("q2", da_t4), ("k1", da_t4), ("k2", da_t4), ("v", da_t4),
                ("lq1", C.c_void_p), ("lk1", C.c_void_p), ("lq2", C.c_void_p), ("lk2", C.c_void_p),
                ("out", da_t4), ("lse1", C.c_void_p), ("lse2", C.c_void_p), ("rstd", C.c_void_p),
                ("o2", da_t4), ("lambda_out", C.c_void_p),
                ("workspace", C.c_void_p), ("workspace_bytes", C.c_size_t), ("rms_weight", C.c_void_p)]


class da_v1_bwd_params(C.Structure):
    _fields_ = [("B", C.c_int), ("N", C.c_int), ("H", C.c_int), ("d_qk", C.c_int), ("d_v", C.c_int),
                ("dtype", C.c_int), ("causal", C.c_int), ("softmax_scale", C.c_float),
                ("lambda_init", C.c_float), ("rms_eps", C.c_float),
                ("q1", da_t4), ("q2", da_t4), ("k1", da_t4), ("k2", da_t4), ("v", da_t4),
                ("lq1", C.c_void_p), ("lk1", C.c_void_p), ("lq2", C.c_void_p), ("lk2", C.c_void_p),
                ("out", da_t4), ("dout", da_t4),
                ("lse1", C.c_void_p), ("lse2", C.c_void_p), ("rstd", C.c_void_p), ("o2", da_t4),
                ("dq1", da_t4), ("dq2", da_t4), ("dk1", da_t4), ("dk2", da_t4), ("dv", da_t4),
                ("dlq1", C.c_void_p), ("dlk1", C.c_void_p), ("dlq2", C.c_void_p), ("dlk2", C.c_void_p),
                ("workspace", C.c_void_p), ("workspace_bytes", C.c_size_t), ("deterministic", C.c_int),
                ("rms_weight", C.c_void_p)]


class da_v1_decode_params(C.Structure):
    _fields_ = [("B", C.c_int), ("H", C.c_int), ("d_qk", C.c_int), ("d_v", C.c_int), ("L_max", C.c_int),
                ("softmax_scale", C.c_float), ("lambda_init", C.c_float), ("rms_eps", C.c_float),
                ("q1", C.c_void_p), ("q2", C.c_void_p), ("k1_cache", da_t4), ("k2_cache", da_t4),
                ("v_cache", da_t4), ("seqlens", C.c_void_p), ("lq1", C.c_void_p), ("lk1", C.c_void_p),
                ("lq2", C.c_void_p), ("lk2", C.c_void_p), ("out", C.c_void_p), ("num_splits", C.c_int),
                ("workspace", C.c_void_p), ("workspace_bytes", C.c_size_t), ("rms_weight", C.c_void_p)]


class da_v2_gate_params(C.Structure):
    _fields_ = [("T", C.c_int), ("d_model", C.c_int), ("h", C.c_int), ("x", C.c_void_p),
                ("x_stride", C.c_int64), ("w_lambda", C.c_void_p), ("gate", C.c_void_p)]


class da_v2_fwd_params(C.Structure):
    _fields_ = [("B", C.c_int), ("N", C.c_int), ("h", C.c_int), ("h_kv", C.c_int), ("d", C.c_int),
                ("d_model", C.c_int), ("causal", C.c_int), ("softmax_scale", C.c_float),
                ("q", da_t4), ("k", da_t4), ("v", da_t4), ("gate", C.c_void_p), ("x", C.c_void_p),
                ("w_lambda", C.c_void_p), ("out", da_t4), ("lse", C.c_void_p), ("o_heads", da_t4),
                ("workspace", C.c_void_p), ("workspace_bytes", C.c_size_t)]


class da_grouped_fwd_params(C.Structure):
    _fields_ = [("B", C.c_int), ("N", C.c_int), ("h", C.c_int), ("ratio", C.c_int), ("h_kv", C.c_int),
                ("d", C.c_int), ("d_model", C.c_int), ("causal", C.c_int), ("softmax_scale", C.c_float),
                ("q", da_t4), ("k", da_t4), ("v", da_t4), ("gate", C.c_void_p), ("x", C.c_void_p),
                ("w_lambda", C.c_void_p), ("out", da_t4), ("lse", C.c_void_p), ("o_heads", da_t4),
                ("workspace", C.c_void_p), ("workspace_bytes", C.c_size_t)]


class da_v2_bwd_params(C.Structure):
    _fields_ = [("B", C.c_int), ("N", C.c_int), ("h", C.c_int), ("h_kv", C.c_int), ("d", C.c_int),
                ("d_model", C.c_int), ("causal", C.c_int), ("softmax_scale", C.c_float),
                ("q", da_t4), ("k", da_t4), ("v", da_t4), ("gate", C.c_void_p), ("x", C.c_void_p),
                ("w_lambda", C.c_void_p), ("o_heads", da_t4), ("lse", C.c_void_p), ("dout", da_t4),
                ("dq", da_t4), ("dk", da_t4), ("dv", da_t4), ("dgate_logit", C.c_void_p),
                ("dx", C.c_void_p), ("dw_lambda", C.c_void_p),
                ("workspace", C.c_void_p), ("workspace_bytes", C.c_size_t)]


class da_grouped_bwd_params(C.Structure):
    _fields_ = [("B", C.c_int), ("N", C.c_int), ("h", C.c_int), ("ratio", C.c_int), ("h_kv", C.c_int),
                ("d", C.c_int), ("d_model", C.c_int), ("causal", C.c_int), ("softmax_scale", C.c_float),
                ("q", da_t4), ("k", da_t4), ("v", da_t4), ("gate", C.c_void_p), ("x", C.c_void_p),
                ("w_lambda", C.c_void_p), ("o_heads", da_t4), ("lse", C.c_void_p), ("dout", da_t4),
                ("dq", da_t4), ("dk", da_t4), ("dv", da_t4), ("dgate_logit", C.c_void_p),
                ("dx", C.c_void_p), ("dw_lambda", C.c_void_p),
                ("workspace", C.c_void_p), ("workspace_bytes", C.c_size_t)]


class da_v2_decode_params(C.Structure):
    _fields_ = [("B", C.c_int), ("h", C.c_int), ("h_kv", C.c_int), ("d", C.c_int),
                ("L_max", C.c_int), ("d_model", C.c_int), ("softmax_scale", C.c_float),
                ("q", C.c_void_p), ("k_cache", da_t4), ("v_cache", da_t4), ("seqlens", C.c_void_p),
                ("gate", C.c_void_p), ("x", C.c_void_p), ("w_lambda", C.c_void_p),
                ("out", C.c_void_p), ("num_splits", C.c_int), ("workspace", C.c_void_p),
                ("workspace_bytes", C.c_size_t)]


class da_kv4_append_params(C.Structure):
    _fields_ = [("B", C.c_int), ("N", C.c_int), ("h_kv", C.c_int), ("d", C.c_int), ("L_max", C.c_int),
                ("k", da_t4), ("v", da_t4), ("cache", da_t4), ("start", C.c_void_p), ("counts", C.c_void_p),
                ("key_weights", C.c_void_p), ("positions", C.c_void_p), ("first_position", C.c_void_p)]


class da_kv4_read_params(C.Structure):
    _fields_ = [("B", C.c_int), ("N", C.c_int), ("h_kv", C.c_int), ("d", C.c_int), ("L_max", C.c_int),
                ("cache", da_t4), ("start", C.c_void_p), ("counts", C.c_void_p), ("k_out", da_t4),
                ("v_out", da_t4)]


class da_v2_decode_kv4_params(C.Structure):
    _fields_ = [("B", C.c_int), ("h", C.c_int), ("h_kv", C.c_int), ("d", C.c_int),
                ("L_max", C.c_int), ("d_model", C.c_int), ("softmax_scale", C.c_float),
                ("q", C.c_void_p), ("cache", da_t4), ("seqlens", C.c_void_p),
                ("gate", C.c_void_p), ("x", C.c_void_p), ("w_lambda", C.c_void_p),
                ("weights_in", C.c_void_p), ("weights_out", C.c_void_p), ("out", C.c_void_p),
                ("workspace", C.c_void_p), ("workspace_bytes", C.c_size_t)]


class da_v2_decode_weighted_params(C.Structure):
    _fields_ = [("decode", da_v2_decode_params), ("weights_in", C.c_void_p), ("weights_out", C.c_void_p)]


DIFFATTN_EVICT_MAX_ROWS = 3


class da_kv_evict_params(C.Structure):
    _fields_ = [("B", C.c_int), ("h_kv", C.c_int), ("L_max", C.c_int), ("keep", C.c_int),
                ("sinks", C.c_int), ("recent", C.c_int), ("seqlens", C.c_void_p),
                ("seqlens_out", C.c_void_p), ("weights_in", C.c_void_p), ("weights_out", C.c_void_p),
                ("positions_in", C.c_void_p), ("positions_out", C.c_void_p), ("next_position", C.c_void_p),
                ("n_rows", C.c_int), ("row_bytes", C.c_int * DIFFATTN_EVICT_MAX_ROWS),
                ("rows", da_t4 * DIFFATTN_EVICT_MAX_ROWS), ("workspace", C.c_void_p),
                ("workspace_bytes", C.c_size_t)]


class da_t3(C.Structure):
    _fields_ = [("ptr", C.c_void_p), ("st", C.c_int64), ("sh", C.c_int64)]


class da_qk_rope_fwd_params(C.Structure):
    _fields_ = [("B", C.c_int), ("N", C.c_int), ("h_q", C.c_int), ("h_k", C.c_int), ("d", C.c_int),
                ("dtype", C.c_int), ("rot_dim", C.c_int), ("interleaved", C.c_int), ("inv_freq", C.c_void_p),
                ("rope_scale", C.c_float), ("norm", C.c_int), ("norm_eps", C.c_float), ("q_weight", C.c_void_p),
                ("k_weight", C.c_void_p), ("positions", C.c_void_p), ("q", da_t4), ("k", da_t4),
                ("q_out", da_t4), ("k_out", da_t4)]


class da_qk_rope_bwd_params(C.Structure):
    _fields_ = [("fwd", da_qk_rope_fwd_params), ("dq_out", da_t4), ("dk_out", da_t4), ("dq", da_t4), ("dk", da_t4),
                ("dq_weight", C.c_void_p), ("dk_weight", C.c_void_p), ("workspace", C.c_void_p),
                ("workspace_bytes", C.c_size_t)]


class da_paged_cache(C.Structure):
    _fields_ = [("B", C.c_int), ("T", C.c_int), ("h_kv", C.c_int), ("d", C.c_int), ("page_size", C.c_int),
                ("n_pages", C.c_int), ("max_pages", C.c_int), ("k_pages", da_t4), ("v_pages", da_t4),
                ("block_table", C.c_void_p), ("cu_seqlens", C.c_void_p), ("seqlens", C.c_void_p)]


class da_paged_append_params(C.Structure):
    _fields_ = [("cache", da_paged_cache), ("h_q", C.c_int), ("rot_dim", C.c_int), ("interleaved", C.c_int),
                ("inv_freq", C.c_void_p), ("rope_scale", C.c_float), ("norm", C.c_int), ("norm_eps", C.c_float),
                ("q_weight", C.c_void_p), ("k_weight", C.c_void_p), ("positions", C.c_void_p), ("k", da_t3),
                ("v", da_t3), ("q", da_t3), ("q_out", da_t3)]


class da_v2_paged_fwd_params(C.Structure):
    _fields_ = [("cache", da_paged_cache), ("h", C.c_int), ("d_model", C.c_int), ("max_new", C.c_int),
                ("softmax_scale", C.c_float), ("q", da_t3), ("gate", C.c_void_p), ("x", C.c_void_p),
                ("w_lambda", C.c_void_p), ("out", da_t3), ("workspace", C.c_void_p), ("workspace_bytes", C.c_size_t)]


_lib = None
_lock = threading.Lock()


def load(path: str = LIB_PATH):
    """Load the shared library once and declare the signatures."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(path):
            raise RuntimeError(
                f"{path} is missing: build it with `python -m differential_attention_diff_gb300.build` "
                "(there is no fallback implementation)")
        lib = C.CDLL(path)
        vp = C.c_void_p
        lib.diffattn_lambda_init.restype = C.c_float
        lib.diffattn_lambda_init.argtypes = [C.c_int]
        lib.diffattn_status_string.restype = C.c_char_p
        lib.diffattn_status_string.argtypes = [C.c_int]
        for name, st in (("diffattn_v1_fwd", da_v1_fwd_params), ("diffattn_v1_bwd", da_v1_bwd_params),
                         ("diffattn_v2_gate", da_v2_gate_params), ("diffattn_v2_fwd", da_v2_fwd_params),
                         ("diffattn_v2_bwd", da_v2_bwd_params), ("diffattn_v1_decode", da_v1_decode_params),
                         ("diffattn_grouped_fwd", da_grouped_fwd_params),
                         ("diffattn_grouped_bwd", da_grouped_bwd_params),
                         ("diffattn_v2_decode", da_v2_decode_params),
                         ("diffattn_v2_decode_noalloc", da_v2_decode_params),
                         ("diffattn_kv4_append", da_kv4_append_params),
                         ("diffattn_kv4_read", da_kv4_read_params),
                         ("diffattn_v2_decode_kv4", da_v2_decode_kv4_params),
                         ("diffattn_v2_decode_weighted", da_v2_decode_weighted_params),
                         ("diffattn_kv_evict", da_kv_evict_params),
                         ("diffattn_qk_rope_fwd", da_qk_rope_fwd_params),
                         ("diffattn_qk_rope_bwd", da_qk_rope_bwd_params),
                         ("diffattn_paged_append", da_paged_append_params),
                         ("diffattn_v2_paged_fwd", da_v2_paged_fwd_params)):
            f = getattr(lib, name)
            f.restype = C.c_int
            f.argtypes = [C.POINTER(st), vp]
        lib.diffattn_v1_fwd_workspace_size.restype = C.c_size_t
        lib.diffattn_v1_fwd_workspace_size.argtypes = [C.c_int] * 6
        lib.diffattn_v1_bwd_workspace_size.restype = C.c_size_t
        lib.diffattn_v1_bwd_workspace_size.argtypes = [C.c_int] * 6
        lib.diffattn_v2_fwd_workspace_size.restype = C.c_size_t
        lib.diffattn_v2_fwd_workspace_size.argtypes = [C.c_int] * 4
        lib.diffattn_v1_decode_num_splits.restype = C.c_int
        lib.diffattn_v1_decode_num_splits.argtypes = [C.c_int] * 3
        lib.diffattn_v1_decode_workspace_size.restype = C.c_size_t
        lib.diffattn_v1_decode_workspace_size.argtypes = [C.c_int] * 5
        lib.diffattn_grouped_fwd_workspace_size.restype = C.c_size_t
        lib.diffattn_grouped_fwd_workspace_size.argtypes = [C.c_int] * 7
        lib.diffattn_grouped_bwd_workspace_size.restype = C.c_size_t
        lib.diffattn_grouped_bwd_workspace_size.argtypes = [C.c_int] * 5
        lib.diffattn_v2_bwd_workspace_size.restype = C.c_size_t
        lib.diffattn_v2_bwd_workspace_size.argtypes = [C.c_int] * 4
        lib.diffattn_v2_decode_num_splits.restype = C.c_int
        lib.diffattn_v2_decode_num_splits.argtypes = [C.c_int] * 3
        lib.diffattn_v2_decode_workspace_size.restype = C.c_size_t
        lib.diffattn_v2_decode_workspace_size.argtypes = [C.c_int] * 7
        lib.diffattn_kv4_record_bytes.restype = C.c_int
        lib.diffattn_kv4_record_bytes.argtypes = [C.c_int]
        for name, n in (("diffattn_v2_decode_kv4_workspace_size", 7),
                        ("diffattn_v2_decode_weighted_workspace_size", 7),
                        ("diffattn_kv_evict_workspace_size", 4),
                        ("diffattn_qk_rope_bwd_workspace_size", 5),
                        ("diffattn_v2_paged_fwd_workspace_size", 7)):
            f = getattr(lib, name)
            f.restype = C.c_size_t
            f.argtypes = [C.c_int] * n
        lib.diffattn_rope_inv_freq.restype = C.c_int
        lib.diffattn_rope_inv_freq.argtypes = [C.c_int, C.c_double, C.c_int, C.c_double, C.c_int,
                                               C.POINTER(C.c_float), C.POINTER(C.c_float)]
        lib.diffattn_debug_inject_fault.restype = C.c_int
        lib.diffattn_debug_inject_fault.argtypes = [C.c_int]
        lib.diffattn_get_device_status.restype = C.c_int
        lib.diffattn_get_device_status.argtypes = [vp]
        lib.diffattn_get_device_status_detail.restype = C.c_int
        lib.diffattn_get_device_status_detail.argtypes = [vp, C.POINTER(C.c_uint32)]
        _lib = lib
        return lib


def _status_str(status: int) -> str:
    try:
        return load().diffattn_status_string(status).decode()
    except Exception:  # noqa: BLE001 - message only
        return "unknown"


def _check(status: int, what: str):
    if status != DA_OK:
        raise DiffAttnError(status, what)


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return C.c_void_p(stream.cuda_stream)


def _t4(t):
    if t is None:
        return da_t4(None, 0, 0, 0)
    if t.dim() != 4 or t.stride(3) != 1:
        raise ValueError("4-D tensor with a contiguous last dimension expected")
    return da_t4(t.data_ptr(), t.stride(0), t.stride(1), t.stride(2))


def _ptr(t):
    return None if t is None else t.data_ptr()


def _dtype_code(t):
    if t.dtype == torch.bfloat16:
        return DA_BF16
    if t.dtype == torch.float32:
        return DA_F32
    raise ValueError(f"unsupported dtype {t.dtype}")


def diffattn_lambda_init(layer: int) -> float:
    return float(load().diffattn_lambda_init(int(layer)))


def diffattn_v1_fwd(q1, q2, k1, k2, v, lq1, lk1, lq2, lk2, lambda_init, *, out=None,
                    causal=True, softmax_scale=0.0, rms_eps=1e-5, rms_weight=None, save=False,
                    saves=None, workspace=None, stream=None):
    """V1 forward.  Returns ``out`` or, with save=True, ``(out, saves)`` where
    saves = dict(lse1, lse2, rstd, o2, lam) are the tensors the backward reads.
    rms_weight: fp32 [d_v] RMSNorm weight (None = unit)."""
    lib = load()
    B, N, H, dqk = q1.shape
    dv = v.shape[-1]
    if out is None:
        out = torch.empty((B, N, H, dv), dtype=v.dtype, device=v.device)
    if save and saves is None:
        f32 = dict(dtype=torch.float32, device=v.device)
        saves = dict(lse1=torch.empty((B, H, N), **f32), lse2=torch.empty((B, H, N), **f32),
                     rstd=torch.empty((B, H, N), **f32),
                     o2=torch.empty((B, N, H, dv), dtype=v.dtype, device=v.device),
                     lam=torch.empty((1,), **f32))
    if not save:
        saves = None
    need = lib.diffattn_v1_fwd_workspace_size(B, N, H, dqk, dv, _dtype_code(q1))
    if workspace is None and need:
        workspace = torch.empty((need,), dtype=torch.uint8, device=v.device)
    p = da_v1_fwd_params(
        B, N, H, dqk, dv, _dtype_code(q1), int(causal), float(softmax_scale), float(lambda_init),
        float(rms_eps), _t4(q1), _t4(q2), _t4(k1), _t4(k2), _t4(v), _ptr(lq1), _ptr(lk1),
        _ptr(lq2), _ptr(lk2), _t4(out),
        _ptr(saves["lse1"]) if saves else None, _ptr(saves["lse2"]) if saves else None,
        _ptr(saves["rstd"]) if saves else None, _t4(saves["o2"] if saves else None),
        _ptr(saves["lam"]) if saves else None, _ptr(workspace),
        0 if workspace is None else workspace.numel() * workspace.element_size(), _ptr(rms_weight))
    _check(lib.diffattn_v1_fwd(C.byref(p), _stream(stream)), "diffattn_v1_fwd")
    return (out, saves) if save else out


def diffattn_v1_bwd(q1, q2, k1, k2, v, lq1, lk1, lq2, lk2, lambda_init, out, dout, saves, *,
                    causal=True, softmax_scale=0.0, rms_eps=1e-5, rms_weight=None, grads=None,
                    workspace=None, deterministic=False, stream=None):
    """V1 backward.  Returns dict(dq1, dq2, dk1, dk2, dv, dlq1, dlk1, dlq2, dlk2).
    deterministic=True makes dQ (and so every output) bitwise reproducible.
    rms_weight: the forward's RMSNorm weight (None = unit; entries nonzero)."""
    lib = load()
    B, N, H, dqk = q1.shape
    dv = v.shape[-1]
    if grads is None:
        grads = {n: torch.empty_like(t) for n, t in
                 (("dq1", q1), ("dq2", q2), ("dk1", k1), ("dk2", k2), ("dv", v),
                  ("dlq1", lq1), ("dlk1", lk1), ("dlq2", lq2), ("dlk2", lk2))}
    need = lib.diffattn_v1_bwd_workspace_size(B, N, H, dqk, dv, int(bool(deterministic)))
    if workspace is None:
        workspace = torch.empty((max(need, 1),), dtype=torch.uint8, device=v.device)
    p = da_v1_bwd_params(
        B, N, H, dqk, dv, _dtype_code(q1), int(causal), float(softmax_scale), float(lambda_init),
        float(rms_eps), _t4(q1), _t4(q2), _t4(k1), _t4(k2), _t4(v), _ptr(lq1), _ptr(lk1),
        _ptr(lq2), _ptr(lk2), _t4(out), _t4(dout), _ptr(saves["lse1"]), _ptr(saves["lse2"]),
        _ptr(saves["rstd"]), _t4(saves["o2"]), _t4(grads["dq1"]), _t4(grads["dq2"]),
        _t4(grads["dk1"]), _t4(grads["dk2"]), _t4(grads["dv"]), _ptr(grads["dlq1"]),
        _ptr(grads["dlk1"]), _ptr(grads["dlq2"]), _ptr(grads["dlk2"]), workspace.data_ptr(),
        workspace.numel() * workspace.element_size(), int(bool(deterministic)), _ptr(rms_weight))
    _check(lib.diffattn_v1_bwd(C.byref(p), _stream(stream)), "diffattn_v1_bwd")
    return grads


def diffattn_v1_decode_num_splits(B, H, L_max) -> int:
    return int(load().diffattn_v1_decode_num_splits(B, H, L_max))


def diffattn_v1_decode_workspace_size(B, H, d_v, L_max, num_splits=0) -> int:
    return int(load().diffattn_v1_decode_workspace_size(B, H, d_v, L_max, num_splits))


def diffattn_v1_decode(q1, q2, k1_cache, k2_cache, v_cache, lq1, lk1, lq2, lk2, lambda_init, *,
                       seqlens=None, out=None, num_splits=0, softmax_scale=0.0, rms_eps=1e-5,
                       rms_weight=None, workspace=None, stream=None):
    """V1 decode: out [B, H, d_v] for one new token per sequence.
    rms_weight: fp32 [d_v] RMSNorm weight (None = unit)."""
    lib = load()
    B, H, dqk = q1.shape
    L_max, dv = v_cache.shape[1], v_cache.shape[3]
    if out is None:
        out = torch.empty((B, H, dv), dtype=q1.dtype, device=q1.device)
    need = lib.diffattn_v1_decode_workspace_size(B, H, dv, L_max, num_splits)
    if workspace is None:
        workspace = torch.empty((max(need, 1),), dtype=torch.uint8, device=q1.device)
    p = da_v1_decode_params(
        B, H, dqk, dv, L_max, float(softmax_scale), float(lambda_init), float(rms_eps), q1.data_ptr(),
        q2.data_ptr(), _t4(k1_cache), _t4(k2_cache), _t4(v_cache), _ptr(seqlens), _ptr(lq1), _ptr(lk1),
        _ptr(lq2), _ptr(lk2), out.data_ptr(), int(num_splits), workspace.data_ptr(),
        workspace.numel() * workspace.element_size(), _ptr(rms_weight))
    _check(lib.diffattn_v1_decode(C.byref(p), _stream(stream)), "diffattn_v1_decode")
    return out


def diffattn_v2_gate(x, w_lambda, *, gate=None, stream=None):
    """gate = sigmoid(x @ w_lambda) for x [..., d_model] -> fp32 [..., h]."""
    lib = load()
    d_model = x.shape[-1]
    h = w_lambda.shape[1]
    x2 = x.reshape(-1, d_model)
    T = x2.shape[0]
    if gate is None:
        gate = torch.empty((*x.shape[:-1], h), dtype=torch.float32, device=x.device)
    p = da_v2_gate_params(T, d_model, h, x2.data_ptr(), x2.stride(0), w_lambda.data_ptr(),
                          gate.data_ptr())
    _check(lib.diffattn_v2_gate(C.byref(p), _stream(stream)), "diffattn_v2_gate")
    return gate


def diffattn_v2_fwd(q, k, v, *, gate=None, x=None, w_lambda=None, out=None, lse=None,
                    causal=True, softmax_scale=0.0, save=False, saves=None, workspace=None,
                    stream=None):
    """V2 forward: out [B, N, h, d] = O_even - gate * O_odd.  With save=True
    returns ``(out, saves)``, saves = dict(lse, o_heads): what the backward reads."""
    lib = load()
    B, N, H2, d = q.shape
    h = H2 // 2
    hkv = k.shape[2]
    if out is None:
        out = torch.empty((B, N, h, d), dtype=q.dtype, device=q.device)
    if save:
        if saves is None:
            saves = dict(lse=torch.empty((B, H2, N), dtype=torch.float32, device=q.device),
                         o_heads=torch.empty((B, N, H2, d), dtype=q.dtype, device=q.device))
        lse = saves["lse"]
    d_model = 0 if x is None else x.shape[-1]
    need = lib.diffattn_v2_fwd_workspace_size(B, N, h, int(gate is not None))
    if workspace is None and need:
        workspace = torch.empty((need,), dtype=torch.uint8, device=q.device)
    p = da_v2_fwd_params(
        B, N, h, hkv, d, d_model, int(causal), float(softmax_scale), _t4(q), _t4(k), _t4(v),
        _ptr(gate), _ptr(x), _ptr(w_lambda), _t4(out), _ptr(lse),
        _t4(saves["o_heads"] if save else None),
        _ptr(workspace), 0 if workspace is None else workspace.numel() * workspace.element_size())
    _check(lib.diffattn_v2_fwd(C.byref(p), _stream(stream)), "diffattn_v2_fwd")
    return (out, saves) if save else out


def diffattn_grouped_fwd(q, k, v, ratio, *, gate=None, x=None, w_lambda=None, out=None, lse=None,
                         o_heads=None, causal=True, softmax_scale=0.0, workspace=None, stream=None):
    """Grouped differential attention: q [B, N, h (ratio+1)/ratio, d] in groups
    of `ratio` signal heads then one noise head; out [B, N, h, d]."""
    lib = load()
    B, N, Hq, d = q.shape
    h = Hq // (ratio + 1) * ratio
    hkv = k.shape[2]
    if out is None:
        out = torch.empty((B, N, h, d), dtype=q.dtype, device=q.device)
    d_model = 0 if x is None else x.shape[-1]
    need = lib.diffattn_grouped_fwd_workspace_size(B, N, h, ratio, d, int(gate is not None),
                                                   int(o_heads is not None))
    if workspace is None and need:
        workspace = torch.empty((need,), dtype=torch.uint8, device=q.device)
    p = da_grouped_fwd_params(
        B, N, h, int(ratio), hkv, d, d_model, int(causal), float(softmax_scale), _t4(q), _t4(k), _t4(v),
        _ptr(gate), _ptr(x), _ptr(w_lambda), _t4(out), _ptr(lse), _t4(o_heads), _ptr(workspace),
        0 if workspace is None else workspace.numel() * workspace.element_size())
    _check(lib.diffattn_grouped_fwd(C.byref(p), _stream(stream)), "diffattn_grouped_fwd")
    return out


def diffattn_v2_bwd_workspace_size(B, N, h, d_model=0) -> int:
    return int(load().diffattn_v2_bwd_workspace_size(B, N, h, d_model))


def diffattn_v2_bwd(q, k, v, dout, saves, *, gate=None, x=None, w_lambda=None, grads=None,
                    want_dx=None, want_dw=None, want_dz=False, causal=True, softmax_scale=0.0,
                    workspace=None, stream=None):
    """V2 backward.  Returns dict(dq, dk, dv) plus dx, dw (when x and w_lambda
    are given, unless want_dx / want_dw say otherwise) and dz (want_dz)."""
    lib = load()
    B, N, H2, d = q.shape
    h = H2 // 2
    hkv = k.shape[2]
    d_model = 0 if x is None else x.shape[-1]
    have_xw = x is not None and w_lambda is not None
    want_dx = have_xw if want_dx is None else want_dx
    want_dw = have_xw if want_dw is None else want_dw
    if grads is None:
        grads = dict(dq=torch.empty_like(q), dk=torch.empty_like(k), dv=torch.empty_like(v))
        if want_dx:
            grads["dx"] = torch.empty((B, N, d_model), dtype=q.dtype, device=q.device)
        if want_dw:
            grads["dw"] = torch.empty((d_model, h), dtype=torch.float32, device=q.device)
        if want_dz:
            grads["dz"] = torch.empty((B, N, h), dtype=torch.float32, device=q.device)
    need = lib.diffattn_v2_bwd_workspace_size(B, N, h, d_model if grads.get("dw") is not None else 0)
    if workspace is None:
        workspace = torch.empty((max(need, 1),), dtype=torch.uint8, device=q.device)
    p = da_v2_bwd_params(
        B, N, h, hkv, d, d_model, int(causal), float(softmax_scale), _t4(q), _t4(k), _t4(v),
        _ptr(gate), _ptr(x), _ptr(w_lambda), _t4(saves["o_heads"]), _ptr(saves["lse"]), _t4(dout),
        _t4(grads["dq"]), _t4(grads["dk"]), _t4(grads["dv"]), _ptr(grads.get("dz")),
        _ptr(grads.get("dx")), _ptr(grads.get("dw")), workspace.data_ptr(),
        workspace.numel() * workspace.element_size())
    _check(lib.diffattn_v2_bwd(C.byref(p), _stream(stream)), "diffattn_v2_bwd")
    return grads


def diffattn_grouped_bwd_workspace_size(B, N, h, ratio, d_model=0) -> int:
    return int(load().diffattn_grouped_bwd_workspace_size(B, N, h, ratio, d_model))


def diffattn_grouped_bwd(q, k, v, dout, saves, ratio, *, gate=None, x=None, w_lambda=None, grads=None,
                         want_dx=None, want_dw=None, want_dz=False, causal=True, softmax_scale=0.0,
                         workspace=None, stream=None):
    """Grouped differential attention backward.  saves: dict(o_heads [B, N, Hq,
    d] bf16, lse [B, Hq, N] fp32) written by diffattn_grouped_fwd.  Returns
    dict(dq, dk, dv) plus dx, dw (when x and w_lambda are given, unless
    want_dx / want_dw say otherwise) and dz (want_dz)."""
    lib = load()
    B, N, Hq, d = q.shape
    h = Hq // (ratio + 1) * ratio
    hkv = k.shape[2]
    d_model = 0 if x is None else x.shape[-1]
    have_xw = x is not None and w_lambda is not None
    want_dx = have_xw if want_dx is None else want_dx
    want_dw = have_xw if want_dw is None else want_dw
    if grads is None:
        grads = dict(dq=torch.empty_like(q), dk=torch.empty_like(k), dv=torch.empty_like(v))
        if want_dx:
            grads["dx"] = torch.empty((B, N, d_model), dtype=q.dtype, device=q.device)
        if want_dw:
            grads["dw"] = torch.empty((d_model, h), dtype=torch.float32, device=q.device)
        if want_dz:
            grads["dz"] = torch.empty((B, N, h), dtype=torch.float32, device=q.device)
    need = lib.diffattn_grouped_bwd_workspace_size(B, N, h, ratio,
                                                   d_model if grads.get("dw") is not None else 0)
    if workspace is None:
        workspace = torch.empty((max(need, 1),), dtype=torch.uint8, device=q.device)
    p = da_grouped_bwd_params(
        B, N, h, int(ratio), hkv, d, d_model, int(causal), float(softmax_scale), _t4(q), _t4(k), _t4(v),
        _ptr(gate), _ptr(x), _ptr(w_lambda), _t4(saves["o_heads"]), _ptr(saves["lse"]), _t4(dout),
        _t4(grads["dq"]), _t4(grads["dk"]), _t4(grads["dv"]), _ptr(grads.get("dz")),
        _ptr(grads.get("dx")), _ptr(grads.get("dw")), workspace.data_ptr(),
        workspace.numel() * workspace.element_size())
    _check(lib.diffattn_grouped_bwd(C.byref(p), _stream(stream)), "diffattn_grouped_bwd")
    return grads


def diffattn_v2_decode_num_splits(B, h_kv, L_max) -> int:
    return int(load().diffattn_v2_decode_num_splits(B, h_kv, L_max))


def diffattn_v2_decode_workspace_size(B, h, h_kv, d, L_max, num_splits=0, gate_given=False) -> int:
    return int(load().diffattn_v2_decode_workspace_size(B, h, h_kv, d, L_max, num_splits,
                                                        int(gate_given)))


def diffattn_v2_decode(q, k_cache, v_cache, *, seqlens=None, gate=None, x=None, w_lambda=None,
                       out=None, num_splits=0, softmax_scale=0.0, workspace=None, stream=None):
    """V2 decode: out [B, h, d] for one new token per sequence."""
    lib = load()
    B, H2, d = q.shape
    h = H2 // 2
    L_max, hkv = k_cache.shape[1], k_cache.shape[2]
    if out is None:
        out = torch.empty((B, h, d), dtype=q.dtype, device=q.device)
    d_model = 0 if x is None else x.shape[-1]
    need = lib.diffattn_v2_decode_workspace_size(B, h, hkv, d, L_max, num_splits,
                                                 int(gate is not None))
    if workspace is None:
        workspace = torch.empty((max(need, 1),), dtype=torch.uint8, device=q.device)
    p = da_v2_decode_params(
        B, h, hkv, d, L_max, d_model, float(softmax_scale), q.data_ptr(), _t4(k_cache),
        _t4(v_cache), _ptr(seqlens), _ptr(gate), _ptr(x), _ptr(w_lambda), out.data_ptr(),
        int(num_splits), workspace.data_ptr(), workspace.numel() * workspace.element_size())
    _check(lib.diffattn_v2_decode(C.byref(p), _stream(stream)), "diffattn_v2_decode")
    return out


def diffattn_v2_decode_noalloc(q, k_cache, v_cache, *, seqlens=None, gate=None, x=None,
                               w_lambda=None, out=None, num_splits=0, softmax_scale=0.0,
                               stream=None):
    """V2 decode through the entry point that takes no workspace (its scratch
    is a fixed array inside the library; see include/diffattn.h)."""
    lib = load()
    B, H2, d = q.shape
    h = H2 // 2
    L_max, hkv = k_cache.shape[1], k_cache.shape[2]
    if out is None:
        out = torch.empty((B, h, d), dtype=q.dtype, device=q.device)
    d_model = 0 if x is None else x.shape[-1]
    p = da_v2_decode_params(
        B, h, hkv, d, L_max, d_model, float(softmax_scale), q.data_ptr(), _t4(k_cache),
        _t4(v_cache), _ptr(seqlens), _ptr(gate), _ptr(x), _ptr(w_lambda), out.data_ptr(),
        int(num_splits), None, 0)
    _check(lib.diffattn_v2_decode_noalloc(C.byref(p), _stream(stream)), "diffattn_v2_decode_noalloc")
    return out


# ---- 4-bit KV cache, gathered key weights, eviction -------------------------
#
# A decode step of a small batch takes a few microseconds on the GPU, so these
# calls pack their parameter structures with struct (a third of the time that
# filling ctypes structures takes); the layout comes from the ctypes classes.

def _codes(t):
    if issubclass(t, C.Structure):
        return "".join(_codes(f) for _, f in t._fields_)
    if issubclass(t, C.Array):
        return _codes(t._type_) * t._length_
    return {C.c_int: "i", C.c_float: "f", C.c_int64: "q", C.c_size_t: "N", C.c_void_p: "P"}[t]


def _packer(t):
    s = struct.Struct("@" + _codes(t) + "0P")  # the trailing 0P pads to the pointers' alignment
    assert s.size == C.sizeof(t), t
    return s.pack


_pack_append, _pack_read = _packer(da_kv4_append_params), _packer(da_kv4_read_params)
_pack_decode_kv4, _pack_weighted = _packer(da_v2_decode_kv4_params), _packer(da_v2_decode_weighted_params)
_pack_evict = _packer(da_kv_evict_params)
_pack_rope_fwd, _pack_rope_bwd = _packer(da_qk_rope_fwd_params), _packer(da_qk_rope_bwd_params)
_pack_paged_append, _pack_paged_fwd = _packer(da_paged_append_params), _packer(da_v2_paged_fwd_params)
_packed_calls = {}


def _call(name, params, stream):
    """Call the entry point `name` with packed parameters on a raw stream."""
    f = _packed_calls.get(name)
    if f is None:
        f = _packed_calls[name] = C.CFUNCTYPE(C.c_int, C.c_char_p, C.c_void_p)((name, load()))
    status = f(params, stream)
    if status:
        _check(status, name)


def _device(t, stream):
    """The device of t, which has to be the current one (the library launches
    there), and the raw stream to launch on."""
    dev = t.get_device()
    if dev < 0 or dev != torch._C._cuda_getDevice():
        raise ValueError(f"tensors on the current CUDA device expected, got {t.device}")
    if stream is None:
        return dev, torch._C._cuda_getCurrentRawStream(dev)
    if stream.device.index != dev:
        raise ValueError(f"a stream of {t.device} expected, got one of {stream.device}")
    return dev, stream.cuda_stream


def _array(t, shape, dtype, dev, name):
    """The data pointer of a contiguous array of the given shape and type on device dev (None: no array)."""
    if t is None:
        return 0
    if t.dtype != dtype or t.shape != shape or not t.is_contiguous() or t.get_device() != dev:
        raise ValueError(f"{name}: contiguous {dtype} {tuple(shape)} on device {dev} expected, got {t.dtype} "
                         f"{tuple(t.shape)} on {t.device}")
    return t.data_ptr()


def _rows4(t, shape, dtype, dev, name):
    """The da_t4 fields of a tensor of the given shape and type on device dev (strides in its elements)."""
    if t.dtype != dtype or t.shape != shape or t.get_device() != dev:
        raise ValueError(f"{name}: {dtype} {tuple(shape)} on device {dev} expected, got {t.dtype} {tuple(t.shape)} "
                         f"on {t.device}")
    sb, sn, sh, sx = t.stride()
    if sx != 1:
        raise ValueError(f"{name}: a contiguous last dimension expected")
    return t.data_ptr(), sb, sn, sh


def _new(make, like, shape, dtype, stream):
    """make (torch.empty or torch.zeros) on the device of `like`, on the stream
    that the call launches on, so that its memory (and its zeros) are ordered
    with the launch."""
    if stream is None:
        return make(shape, dtype=dtype, device=like.device)
    with torch.cuda.stream(stream):
        return make(shape, dtype=dtype, device=like.device)


@functools.lru_cache(maxsize=4096)
def _need(dev, name, *args):
    """The workspace_size entry point `name`; a function of its arguments and the (current) device dev."""
    return getattr(load(), name)(*args)


def _space(workspace, dev):
    """(pointer, bytes) of a workspace; None is none."""
    if workspace is None:
        return 0, 0
    if workspace.get_device() != dev or not workspace.is_contiguous():
        raise ValueError(f"workspace: a contiguous tensor on device {dev} expected")
    return workspace.data_ptr(), workspace.nbytes


def diffattn_kv4_record_bytes(d) -> int:
    """Bytes of one 4-bit record (a key and a value row): d + 16, 0 if d is unsupported."""
    return int(load().diffattn_kv4_record_bytes(int(d)))


def diffattn_kv4_append(k, v, cache, *, start=None, counts=None, key_weights=None, positions=None,
                        first_position=None, stream=None):
    """Quantise k, v [B, N, h_kv, d] (bf16) into the 4-bit cache, uint8 [B,
    L_max, h_kv, d + 16] in any stride order: row i < counts[b] goes to
    position start[b] + i.  key_weights / positions [B, h_kv, L_max] are reset
    for the written positions."""
    dev, raw = _device(k, stream)
    B, N, hkv, d = shape = k.shape
    L_max, bf16, i32 = cache.shape[1], torch.bfloat16, torch.int32
    per_slot = (B, hkv, L_max)
    _call("diffattn_kv4_append", _pack_append(
        B, N, hkv, d, L_max, *_rows4(k, shape, bf16, dev, "k"), *_rows4(v, shape, bf16, dev, "v"),
        *_rows4(cache, (B, L_max, hkv, d + 16), torch.uint8, dev, "cache"), _array(start, (B,), i32, dev, "start"),
        _array(counts, (B,), i32, dev, "counts"), _array(key_weights, per_slot, torch.float32, dev, "key_weights"),
        _array(positions, per_slot, i32, dev, "positions"),
        _array(first_position, (B,), i32, dev, "first_position")), raw)
    return cache


def diffattn_kv4_read(cache, N, *, start=None, counts=None, k_out=None, v_out=None, stream=None):
    """Positions start[b] .. start[b] + counts[b] - 1 of the 4-bit cache as
    bf16 rows: (k, v) [B, N, h_kv, d].  Rows i >= counts[b] are left as they
    were (zeros where the outputs are allocated here)."""
    dev, raw = _device(cache, stream)
    B, L_max, hkv, rec = cache.shape
    d, bf16 = rec - 16, torch.bfloat16
    shape = (B, N, hkv, d)
    if k_out is None:
        k_out = _new(torch.zeros, cache, shape, bf16, stream)
    if v_out is None:
        v_out = _new(torch.zeros, cache, shape, bf16, stream)
    _call("diffattn_kv4_read", _pack_read(
        B, N, hkv, d, L_max, *_rows4(cache, (B, L_max, hkv, rec), torch.uint8, dev, "cache"),
        _array(start, (B,), torch.int32, dev, "start"), _array(counts, (B,), torch.int32, dev, "counts"),
        *_rows4(k_out, shape, bf16, dev, "k_out"), *_rows4(v_out, shape, bf16, dev, "v_out")), raw)
    return k_out, v_out


def _gate_source(gate, x, w_lambda, B, h, dev):
    """The checked gate or (x, w_lambda) of a decode step: (gate, x, w_lambda, d_model)."""
    if gate is not None:
        return _array(gate, (B, h), torch.float32, dev, "gate"), 0, 0, 0
    if x is None or w_lambda is None:
        return 0, 0, 0, 0  # refused by the library
    d_model = x.shape[-1]
    return (0, _array(x, (B, d_model), torch.bfloat16, dev, "x"),
            _array(w_lambda, (d_model, h), torch.bfloat16, dev, "w_lambda"), d_model)


def diffattn_v2_decode_kv4_workspace_size(B, h, h_kv, d, L_max, gate_given=False, weights=False) -> int:
    return int(load().diffattn_v2_decode_kv4_workspace_size(B, h, h_kv, d, L_max, int(gate_given), int(weights)))


def diffattn_v2_decode_kv4(q, cache, *, seqlens=None, gate=None, x=None, w_lambda=None, weights_in=None,
                           weights_out=None, out=None, softmax_scale=0.0, workspace=None, stream=None):
    """V2 decode over a 4-bit cache (uint8 [B, L_max, h_kv, d + 16]): out [B,
    h, d].  weights_out [B, h_kv, L_max]: weights_in (None = 0, may be the same
    tensor) plus what each key contributes to this step's differential maps."""
    dev, raw = _device(q, stream)
    B, H2, d = q.shape
    L_max, hkv = cache.shape[1], cache.shape[2]
    h, bf16, f32 = H2 // 2, torch.bfloat16, torch.float32
    if out is None:
        out = _new(torch.empty, q, (B, h, d), bf16, stream)
    if workspace is None:
        need = _need(dev, "diffattn_v2_decode_kv4_workspace_size", B, h, hkv, d, L_max, gate is not None,
                     weights_out is not None)
        if need:
            workspace = _new(torch.empty, q, (need,), torch.uint8, stream)
    gate_, x_, w_, d_model = _gate_source(gate, x, w_lambda, B, h, dev)
    per_slot = (B, hkv, L_max)
    _call("diffattn_v2_decode_kv4", _pack_decode_kv4(
        B, h, hkv, d, L_max, d_model, softmax_scale, _array(q, (B, 2 * h, d), bf16, dev, "q"),
        *_rows4(cache, (B, L_max, hkv, d + 16), torch.uint8, dev, "cache"),
        _array(seqlens, (B,), torch.int32, dev, "seqlens"), gate_, x_, w_,
        _array(weights_in, per_slot, f32, dev, "weights_in"), _array(weights_out, per_slot, f32, dev, "weights_out"),
        _array(out, (B, h, d), bf16, dev, "out"), *_space(workspace, dev)), raw)
    return out


def diffattn_v2_decode_weighted_workspace_size(B, h, h_kv, d, L_max, num_splits=0, gate_given=False) -> int:
    return int(load().diffattn_v2_decode_weighted_workspace_size(B, h, h_kv, d, L_max, num_splits,
                                                                 int(gate_given)))


def diffattn_v2_decode_weighted(q, k_cache, v_cache, *, weights_out, weights_in=None, seqlens=None, gate=None,
                                x=None, w_lambda=None, out=None, num_splits=0, softmax_scale=0.0,
                                workspace=None, stream=None):
    """diffattn_v2_decode that also gathers the keys' weights into weights_out
    [B, h_kv, L_max] (see diffattn_v2_decode_kv4)."""
    dev, raw = _device(q, stream)
    B, H2, d = q.shape
    L_max, hkv = k_cache.shape[1], k_cache.shape[2]
    h, bf16, f32 = H2 // 2, torch.bfloat16, torch.float32
    if out is None:
        out = _new(torch.empty, q, (B, h, d), bf16, stream)
    if workspace is None:
        need = _need(dev, "diffattn_v2_decode_weighted_workspace_size", B, h, hkv, d, L_max, num_splits,
                     gate is not None)
        workspace = _new(torch.empty, q, (max(need, 1),), torch.uint8, stream)
    gate_, x_, w_, d_model = _gate_source(gate, x, w_lambda, B, h, dev)
    rows, per_slot = (B, L_max, hkv, d), (B, hkv, L_max)
    _call("diffattn_v2_decode_weighted", _pack_weighted(
        B, h, hkv, d, L_max, d_model, softmax_scale, _array(q, (B, 2 * h, d), bf16, dev, "q"),
        *_rows4(k_cache, rows, bf16, dev, "k_cache"), *_rows4(v_cache, rows, bf16, dev, "v_cache"),
        _array(seqlens, (B,), torch.int32, dev, "seqlens"), gate_, x_, w_, _array(out, (B, h, d), bf16, dev, "out"),
        num_splits, *_space(workspace, dev), _array(weights_in, per_slot, f32, dev, "weights_in"),
        _array(weights_out, per_slot, f32, dev, "weights_out")), raw)
    return out


def diffattn_kv_evict_workspace_size(B, h_kv, L_max, keep) -> int:
    return int(load().diffattn_kv_evict_workspace_size(B, h_kv, L_max, keep))


def diffattn_kv_evict(rows, key_weights, keep, *, sinks=0, recent=0, seqlens=None, positions=None,
                      next_position=None, weights_out=None, positions_out=None, seqlens_out=None,
                      workspace=None, stream=None):
    """Cut the caches in `rows` (up to three tensors [B, L_max, h_kv, width],
    compacted in place) down to the `keep` slots per sequence and KV head that
    gathered the most weight; the first `sinks` and the newest `recent` token
    positions always stay.  Returns dict(key_weights, positions, seqlens) after
    the cut.  Without the _out arguments the given key_weights, positions and
    seqlens are updated in place (a seqlens of None gives a new tensor)."""
    dev, raw = _device(key_weights, stream)
    B, hkv, L_max = shape = key_weights.shape
    i32, f32 = torch.int32, torch.float32
    if not 1 <= len(rows) <= DIFFATTN_EVICT_MAX_ROWS:
        raise ValueError(f"1 to {DIFFATTN_EVICT_MAX_ROWS} caches expected, got {len(rows)}")
    if weights_out is None:
        weights_out = key_weights
    if positions_out is None:
        positions_out = positions
    if seqlens_out is None:
        seqlens_out = _new(torch.empty, key_weights, (B,), i32, stream) if seqlens is None else seqlens
    if workspace is None:
        need = _need(dev, "diffattn_kv_evict_workspace_size", B, hkv, L_max, keep)
        workspace = _new(torch.empty, key_weights, (max(need, 1),), torch.uint8, stream)
    row_bytes, views = [0] * DIFFATTN_EVICT_MAX_ROWS, [0] * (4 * DIFFATTN_EVICT_MAX_ROWS)
    for i, r in enumerate(rows):
        n, width = r.element_size(), r.shape[-1]
        ptr, sb, sn, sh = _rows4(r, (B, L_max, hkv, width), r.dtype, dev, f"rows[{i}]")
        row_bytes[i] = width * n
        views[4 * i:4 * i + 4] = ptr, sb * n, sn * n, sh * n
    _call("diffattn_kv_evict", _pack_evict(
        B, hkv, L_max, keep, sinks, recent, _array(seqlens, (B,), i32, dev, "seqlens"),
        _array(seqlens_out, (B,), i32, dev, "seqlens_out"), _array(key_weights, shape, f32, dev, "key_weights"),
        _array(weights_out, shape, f32, dev, "weights_out"), _array(positions, shape, i32, dev, "positions"),
        _array(positions_out, shape, i32, dev, "positions_out"),
        _array(next_position, (B,), i32, dev, "next_position"), len(rows), *row_bytes, *views,
        *_space(workspace, dev)), raw)
    return dict(key_weights=weights_out, positions=positions_out, seqlens=seqlens_out)


# ---- positions, paged cache --------------------------------------------------

DA_ROPE_STRETCH = {None: 0, "linear": 1, "base": 2, "ramp": 3}


def diffattn_rope_inv_freq(rot_dim, base=10000.0, *, stretch=None, factor=1.0, trained_len=0, device="cuda"):
    """(inv_freq, rope_scale): fp32 [rot_dim / 2] frequencies in radians per position on `device`, and the scale
    of the rotated features, for contexts `factor` times as long as trained (stretch: None, "linear", "base" or
    "ramp", which needs the trained_len in positions)."""
    if stretch not in DA_ROPE_STRETCH:
        raise ValueError(f"stretch: one of {list(DA_ROPE_STRETCH)} expected, got {stretch!r}")
    f, s = (C.c_float * max(rot_dim // 2, 1))(), C.c_float()
    _check(load().diffattn_rope_inv_freq(rot_dim, base, DA_ROPE_STRETCH[stretch], factor, trained_len, f, C.byref(s)),
           "diffattn_rope_inv_freq")
    return torch.tensor(list(f), dtype=torch.float32).to(device), s.value


def _rope_fields(d, inv_freq, rot_dim, interleaved, rope_scale, norm, norm_eps, q_weight, k_weight, dev):
    """The rotation's and the norm's fields, from rot_dim to k_weight."""
    if rot_dim is None:
        rot_dim = 0 if inv_freq is None else 2 * inv_freq.shape[0]
    f32 = torch.float32
    return (rot_dim, interleaved, _array(inv_freq, (rot_dim // 2,), f32, dev, "inv_freq"), rope_scale, norm, norm_eps,
            0 if q_weight is None else _array(q_weight, (d,), f32, dev, "q_weight"),
            0 if k_weight is None else _array(k_weight, (d,), f32, dev, "k_weight"))


_NO_T4, _NO_T3 = (0, 0, 0, 0), (0, 0, 0)


def _out(like, stream):
    """A new contiguous tensor of the shape and type of `like`, on the stream that the call launches on (empty_like:
    1.4 us on the host, new_empty 3.8)."""
    if stream is None:
        return torch.empty_like(like, memory_format=torch.contiguous_format)
    with torch.cuda.stream(stream):
        return torch.empty_like(like, memory_format=torch.contiguous_format)


def _heads4(t, B, N, d, dtype, dev, name, heads=None):
    """The da_t4 fields of a tensor [B, N, heads, d], of any heads where None; none of a tensor that is None."""
    if t is None:
        if heads:
            raise ValueError(f"{name}: a tensor of {heads} heads expected, got None")
        return _NO_T4
    return _rows4(t, (B, N, t.shape[2] if heads is None else heads, d), dtype, dev, name)


def diffattn_qk_rope_fwd(q, k, inv_freq, *, positions=None, rot_dim=None, interleaved=False, rope_scale=1.0, norm=False,
                         norm_eps=1e-5, q_weight=None, k_weight=None, q_out=None, k_out=None, stream=None):
    """Queries [B, N, h_q, d] and keys [B, N, h_k, d] (bf16 or fp32; either may be None) normed per head (norm; fp32
    [d] weights, None = unit) and their first rot_dim (None = all that inv_freq has) features rotated by their
    positions (int32 [B, N], None = 0 .. N-1).  Returns (q_out, k_out), which may be q and k themselves."""
    some = k if q is None else q
    dev, raw = _device(some, stream)
    B, N, _, d = some.shape
    dtype = some.dtype
    h_q = h_k = 0
    if q is not None:
        h_q = q.shape[2]
        if q_out is None:
            q_out = _out(q, stream)
    if k is not None:
        h_k = k.shape[2]
        if k_out is None:
            k_out = _out(k, stream)
    _call("diffattn_qk_rope_fwd", _pack_rope_fwd(
        B, N, h_q, h_k, d, _dtype_code(some),
        *_rope_fields(d, inv_freq, rot_dim, interleaved, rope_scale, norm, norm_eps, q_weight, k_weight, dev),
        0 if positions is None else _array(positions, (B, N), torch.int32, dev, "positions"),
        *_heads4(q, B, N, d, dtype, dev, "q"), *_heads4(k, B, N, d, dtype, dev, "k"),
        *_heads4(q_out, B, N, d, dtype, dev, "q_out", h_q), *_heads4(k_out, B, N, d, dtype, dev, "k_out", h_k)), raw)
    return q_out, k_out


def diffattn_qk_rope_bwd_workspace_size(B, N, h_q, h_k, d) -> int:
    return int(load().diffattn_qk_rope_bwd_workspace_size(B, N, h_q, h_k, d))


def diffattn_qk_rope_bwd(q, k, dq_out, dk_out, inv_freq, *, positions=None, rot_dim=None, interleaved=False,
                         rope_scale=1.0, norm=False, norm_eps=1e-5, q_weight=None, k_weight=None, dq=None, dk=None,
                         dq_weight=None, dk_weight=None, want_weights=None, workspace=None, stream=None):
    """Gradients of diffattn_qk_rope_fwd given those of its outputs: dict(dq, dk) and, with norm (unless want_weights
    is False), dq_weight and dk_weight, fp32 [d].  q and k are needed with norm only.  dq and dk may be dq_out and
    dk_out themselves."""
    some = dk_out if dq_out is None else dq_out
    dev, raw = _device(some, stream)
    B, N, _, d = some.shape
    dtype, f32 = some.dtype, torch.float32
    h_q = h_k = 0
    want = norm if want_weights is None else want_weights
    if dq_out is not None:
        h_q = dq_out.shape[2]
        if dq is None:
            dq = _out(dq_out, stream)
        if want and dq_weight is None:
            dq_weight = _new(torch.empty, some, (d,), f32, stream)
    if dk_out is not None:
        h_k = dk_out.shape[2]
        if dk is None:
            dk = _out(dk_out, stream)
        if want and dk_weight is None:
            dk_weight = _new(torch.empty, some, (d,), f32, stream)
    if workspace is None and (dq_weight is not None or dk_weight is not None):
        need = _need(dev, "diffattn_qk_rope_bwd_workspace_size", B, N, h_q, h_k, d)
        workspace = _new(torch.empty, some, (max(need, 1),), torch.uint8, stream)
    _call("diffattn_qk_rope_bwd", _pack_rope_bwd(
        B, N, h_q, h_k, d, _dtype_code(some),
        *_rope_fields(d, inv_freq, rot_dim, interleaved, rope_scale, norm, norm_eps, q_weight, k_weight, dev),
        0 if positions is None else _array(positions, (B, N), torch.int32, dev, "positions"),
        *(_heads4(q, B, N, d, dtype, dev, "q", h_q) if norm else _NO_T4),
        *(_heads4(k, B, N, d, dtype, dev, "k", h_k) if norm else _NO_T4), *_NO_T4, *_NO_T4,
        *_heads4(dq_out, B, N, d, dtype, dev, "dq_out"), *_heads4(dk_out, B, N, d, dtype, dev, "dk_out"),
        *_heads4(dq, B, N, d, dtype, dev, "dq", h_q), *_heads4(dk, B, N, d, dtype, dev, "dk", h_k),
        0 if dq_weight is None else _array(dq_weight, (d,), f32, dev, "dq_weight"),
        0 if dk_weight is None else _array(dk_weight, (d,), f32, dev, "dk_weight"), *_space(workspace, dev)), raw)
    return dict(dq=dq, dk=dk, dq_weight=dq_weight, dk_weight=dk_weight)


def _rows3(t, shape, dtype, dev, name):
    """The da_t3 fields of a packed tensor of the given shape and type on device dev."""
    if t.dtype != dtype or t.shape != shape or t.get_device() != dev:
        raise ValueError(f"{name}: {dtype} {tuple(shape)} on device {dev} expected, got {t.dtype} {tuple(t.shape)} "
                         f"on {t.device}")
    st, sh, sx = t.stride()
    if sx != 1:
        raise ValueError(f"{name}: a contiguous last dimension expected")
    return t.data_ptr(), st, sh


def _paged_fields(T, k_pages, v_pages, block_table, cu_seqlens, seqlens, dev):
    """The fields of a da_paged_cache."""
    n_pages, page_size, hkv, d = shape = k_pages.shape
    B, max_pages = block_table.shape
    i32 = torch.int32
    return (B, T, hkv, d, page_size, n_pages, max_pages, *_rows4(k_pages, shape, torch.bfloat16, dev, "k_pages"),
            *_rows4(v_pages, shape, torch.bfloat16, dev, "v_pages"),
            _array(block_table, (B, max_pages), i32, dev, "block_table"),
            _array(cu_seqlens, (B + 1,), i32, dev, "cu_seqlens"), _array(seqlens, (B,), i32, dev, "seqlens"))


def diffattn_paged_append(k, v, k_pages, v_pages, block_table, cu_seqlens, seqlens, inv_freq, *, q=None, q_out=None,
                          positions=None, rot_dim=None, interleaved=False, rope_scale=1.0, norm=False, norm_eps=1e-5,
                          q_weight=None, k_weight=None, stream=None):
    """Put new tokens' keys (normed and rotated) and values [T, h_kv, d] into a paged cache: k_pages, v_pages
    [n_pages, page_size, h_kv, d] in any stride order, block_table int32 [B, max_pages].  Sequence b's tokens are
    rows cu_seqlens[b] .. cu_seqlens[b + 1] - 1, the last of its seqlens[b] positions.  q [T, h_q, d] of the same
    tokens goes, normed and rotated too, to q_out (None: a new tensor, whose rows without a sequence are zeros).
    Returns q_out."""
    dev, raw = _device(k, stream)
    T, hkv, d = shape = k.shape
    bf16 = torch.bfloat16
    h_q = 0
    if q is not None:
        h_q = q.shape[1]
        if q_out is None:
            q_out = _new(torch.zeros, q, q.shape, bf16, stream)
    _call("diffattn_paged_append", _pack_paged_append(
        *_paged_fields(T, k_pages, v_pages, block_table, cu_seqlens, seqlens, dev), h_q,
        *_rope_fields(d, inv_freq, rot_dim, interleaved, rope_scale, norm, norm_eps, q_weight, k_weight, dev),
        0 if positions is None else _array(positions, (T,), torch.int32, dev, "positions"),
        *_rows3(k, (T, k_pages.shape[2], k_pages.shape[3]), bf16, dev, "k"),
        *_rows3(v, shape, bf16, dev, "v"), *(_NO_T3 if q is None else _rows3(q, (T, h_q, d), bf16, dev, "q")),
        *(_NO_T3 if q is None else _rows3(q_out, (T, h_q, d), bf16, dev, "q_out"))), raw)
    return q_out


def diffattn_v2_paged_fwd_workspace_size(T, B, max_new, h, h_kv, d, gate_given=False) -> int:
    return int(load().diffattn_v2_paged_fwd_workspace_size(T, B, max_new, h, h_kv, d, int(gate_given)))


def diffattn_v2_paged_fwd(q, k_pages, v_pages, block_table, cu_seqlens, seqlens, *, max_new=0, gate=None, x=None,
                          w_lambda=None, out=None, softmax_scale=0.0, workspace=None, stream=None):
    """V2 attention of new tokens q [T, 2h, d] over a paged cache (see diffattn_paged_append) that holds their keys:
    out [T, h, d] (None: a new tensor, whose rows without a sequence are zeros).  max_new: the most new tokens that
    a sequence is expected to have (0 = T); the kernel is chosen by it: say 1 for a batch of decode steps."""
    dev, raw = _device(q, stream)
    T, H2, d = q.shape
    h, bf16 = H2 // 2, torch.bfloat16
    B, hkv = block_table.shape[0], k_pages.shape[2]
    if out is None:
        out = _new(torch.zeros, q, (T, h, d), bf16, stream)
    if workspace is None:
        need = _need(dev, "diffattn_v2_paged_fwd_workspace_size", T, B, max_new, h, hkv, d, gate is not None)
        workspace = _new(torch.empty, q, (max(need, 1),), torch.uint8, stream)
    gate_, x_, w_, d_model = _gate_source(gate, x, w_lambda, T, h, dev)
    _call("diffattn_v2_paged_fwd", _pack_paged_fwd(
        *_paged_fields(T, k_pages, v_pages, block_table, cu_seqlens, seqlens, dev), h, d_model, max_new, softmax_scale,
        *_rows3(q, (T, 2 * h, k_pages.shape[3]), bf16, dev, "q"), gate_, x_, w_, *_rows3(out, (T, h, d), bf16, dev, "out"),
        *_space(workspace, dev)), raw)
    return out


DA_FAULT_NONE, DA_FAULT_V2_FWD_SKIP_LOAD = 0, 1


def diffattn_debug_inject_fault(fault: int):
    """Test hook: arm a one-shot fault for the next call it applies to."""
    _check(load().diffattn_debug_inject_fault(int(fault)), "diffattn_debug_inject_fault")


def diffattn_get_device_status(stream=None, detail=False):
    lib = load()
    if detail:
        raw = C.c_uint32(0)
        st = lib.diffattn_get_device_status_detail(_stream(stream), C.byref(raw))
        return st, raw.value
    return lib.diffattn_get_device_status(_stream(stream))
