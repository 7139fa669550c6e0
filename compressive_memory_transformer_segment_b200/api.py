"""Thin Python binding of libinfini_attn.so (argument marshalling only).

Every step of the layer runs in the library's CUDA kernels; this module only
checks tensor metadata, builds the C structs and passes raw pointers and the
current CUDA stream.  PyTorch provides device memory and streams.  There is no
fallback: if the library is missing, every call raises.

Names follow the C ABI in include/infini_attn.h.
"""

import ctypes
import functools
import os
from typing import NamedTuple, Optional

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libinfini_attn.so")

RULES = {"linear": 0, "delta": 1}
DTYPES = {torch.bfloat16: 0, torch.float32: 1}
PATHS = {0: "simt", 1: "tcgen05"}

OK = 0
ERR_ARG, ERR_UNSUPPORTED, ERR_ALIAS, ERR_CUDA, ERR_TIMEOUT, ERR_WORKSPACE, ERR_ALIGN = (
    -1, -2, -3, -4, -5, -6, -7)
ERR_SCRATCH_LIMIT = -8
ERR_RANGE = -9


class Dims(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("H_q", ctypes.c_int), ("H_kv", ctypes.c_int),
                ("L", ctypes.c_int), ("d_k", ctypes.c_int), ("d_v", ctypes.c_int),
                ("dtype", ctypes.c_int)]


class Plan(ctypes.Structure):
    _fields_ = [("path", ctypes.c_int), ("launches", ctypes.c_int),
                ("num_segments", ctypes.c_int), ("workspace_bytes", ctypes.c_size_t)]


class _CacheQ4Ptrs(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("k_codes", "k_scale", "v_codes", "v_scale")]


class InfiniError(RuntimeError):
    def __init__(self, status, message):
        super().__init__(f"infini_attn status {status}: {message}")
        self.status = status


_lib = None

# (name, restype, argtypes) for every entry point of include/infini_attn.h.
_P = ctypes.c_void_p
_SIGNATURES = [
    ("infini_attn_version", ctypes.c_int, []),
    ("infini_attn_status_string", ctypes.c_char_p, [ctypes.c_int]),
    ("infini_attn_init_state", ctypes.c_int, [_P, _P, ctypes.c_int, ctypes.c_int, ctypes.c_int,
                                              ctypes.c_int, _P]),
    ("infini_attn_workspace_bytes", ctypes.c_size_t, [ctypes.POINTER(Dims), ctypes.c_int, ctypes.c_int]),
    ("infini_attn_plan", ctypes.c_int, [ctypes.POINTER(Dims), ctypes.c_int, ctypes.c_int,
                                        ctypes.POINTER(Plan)]),
    ("infini_attn_forward", ctypes.c_int, [_P, _P, _P, _P, _P, _P, ctypes.c_int, ctypes.c_int,
                                           ctypes.POINTER(Dims), _P, _P, _P, _P, ctypes.c_size_t, _P]),
    ("infini_attn_state_update", ctypes.c_int, [_P, _P, _P, _P, ctypes.c_int, ctypes.c_int,
                                                ctypes.POINTER(Dims), _P, _P, _P, ctypes.c_size_t, _P]),
    ("infini_attn_state_sum", ctypes.c_int, [_P, _P, _P, ctypes.c_int, ctypes.c_int, ctypes.c_int,
                                             ctypes.c_int, ctypes.c_int, _P, _P, _P]),
    ("infini_attn_decode_workspace_bytes", ctypes.c_size_t, [ctypes.POINTER(Dims), ctypes.c_int,
                                                              ctypes.c_int]),
    ("infini_attn_decode_step", ctypes.c_int, [_P, _P, _P, _P, _P, _P, ctypes.c_int, _P, _P,
                                               ctypes.c_int, ctypes.c_int, ctypes.POINTER(Dims), _P,
                                               _P, ctypes.c_size_t, _P]),
    ("infini_attn_host_arena_bytes", ctypes.c_size_t, [ctypes.POINTER(Dims), ctypes.c_int, ctypes.c_int]),
    ("infini_attn_forward_host", ctypes.c_int, [_P, _P, _P, _P, _P, _P, ctypes.c_int, ctypes.c_int,
                                                ctypes.POINTER(Dims), _P, _P, _P, _P,
                                                ctypes.c_size_t, _P]),
    ("infini_attn_sync_status", ctypes.c_int, [_P]),
    ("infini_attn_set_kernel_timing", ctypes.c_int, [ctypes.c_int]),
    ("infini_attn_kernel_times", ctypes.c_int, [ctypes.POINTER(ctypes.c_double),
                                                ctypes.POINTER(ctypes.c_int), ctypes.c_int,
                                                ctypes.c_int]),
    ("infini_attn_selftest_approx", ctypes.c_int, [_P, _P, _P, _P, ctypes.c_int, _P]),
    ("infini_attn_selftest_timeout", ctypes.c_int, [_P]),
    ("infini_attn_forward_noalloc", ctypes.c_int, [_P, _P, _P, _P, _P, _P, ctypes.c_int,
                                                   ctypes.c_int, ctypes.POINTER(Dims), _P, _P, _P,
                                                   _P]),
    ("infini_attn_noalloc_scratch_limit", ctypes.c_size_t, []),
    ("infini_attn_backward_workspace_bytes", ctypes.c_size_t, [ctypes.POINTER(Dims), ctypes.c_int,
                                                                ctypes.c_int]),
    ("infini_attn_qkv_project", ctypes.c_int, [_P, _P, _P, _P, _P, ctypes.POINTER(Dims), ctypes.c_int,
                                               _P, _P, _P, _P]),
    ("infini_attn_rope_tables", ctypes.c_int, [_P, _P, ctypes.c_int, ctypes.c_int, ctypes.c_double,
                                               _P]),
    ("infini_attn_block_norm", ctypes.c_int, [_P, _P, _P, _P, _P, _P, ctypes.c_float,
                                              ctypes.c_longlong, ctypes.c_int, ctypes.c_int,
                                              _P, _P, _P, _P, _P]),
    ("infini_attn_block_norm_backward_workspace_bytes", ctypes.c_size_t, [ctypes.c_longlong,
                                                                           ctypes.c_int]),
    ("infini_attn_block_norm_backward", ctypes.c_int, [_P] * 10 + [ctypes.c_longlong, ctypes.c_int,
                                                                   ctypes.c_int] + [_P] * 7 +
     [ctypes.c_size_t, _P]),
    ("infini_attn_w4_quantize", ctypes.c_int, [_P] + [ctypes.c_int] * 4 + [_P] * 4),
    ("infini_attn_w4_pack", ctypes.c_int, [_P, ctypes.c_int, ctypes.c_int, _P, _P]),
    ("infini_attn_w4_dequantize", ctypes.c_int, [_P] * 3 + [ctypes.c_int] * 4 + [_P] * 2),
    ("infini_attn_linear_w4", ctypes.c_int, [_P] * 5 + [ctypes.c_int] * 5 + [_P] * 2),
    ("infini_attn_qkv_project_w4", ctypes.c_int, [_P] * 7 + [ctypes.c_int, _P, ctypes.POINTER(Dims),
                                                             ctypes.c_int, ctypes.c_int] + [_P] * 4),
    ("infini_attn_cache_q4_append", ctypes.c_int, [_P, _P, _P, ctypes.POINTER(Dims), ctypes.c_int,
                                                   ctypes.POINTER(_CacheQ4Ptrs), _P]),
    ("infini_attn_cache_q4_read", ctypes.c_int, [ctypes.POINTER(_CacheQ4Ptrs), ctypes.POINTER(Dims),
                                                 ctypes.c_int, _P, _P, _P]),
    ("infini_attn_state_update_q4_workspace_bytes", ctypes.c_size_t, [ctypes.POINTER(Dims),
                                                                      ctypes.c_int]),
    ("infini_attn_state_update_q4", ctypes.c_int, [ctypes.POINTER(_CacheQ4Ptrs), _P, _P, ctypes.c_int,
                                                   ctypes.POINTER(Dims), ctypes.c_int, _P, _P, _P,
                                                   ctypes.c_size_t, _P]),
    ("infini_attn_decode_q4_workspace_bytes", ctypes.c_size_t, [ctypes.POINTER(Dims), ctypes.c_int]),
    ("infini_attn_decode_step_q4", ctypes.c_int, [_P, _P, _P, _P, ctypes.POINTER(_CacheQ4Ptrs), _P, _P,
                                                  _P, ctypes.c_int, ctypes.POINTER(Dims), _P, _P,
                                                  ctypes.c_size_t, _P]),
    ("infini_attn_backward", ctypes.c_int, [_P, _P, _P, _P, _P, _P, ctypes.c_int, ctypes.c_int,
                                            ctypes.POINTER(Dims), _P, _P, _P, _P, _P, _P, _P, _P,
                                            _P, _P, ctypes.c_size_t, _P]),
]


def load_library(path=None):
    """Load the in-tree CUDA library (raises if it was not built)."""
    global _lib
    if _lib is not None:
        return _lib
    path = path or LIB_PATH
    if not os.path.exists(path):
        raise FileNotFoundError(
            f"{path} is missing: build it with "
            "`python -m compressive_memory_transformer_segment_b200.build`")
    lib = ctypes.CDLL(path)
    for name, res, args in _SIGNATURES:
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    _lib = lib
    return lib


def exported_symbols():
    return [name for name, _, _ in _SIGNATURES]


def status_string(status):
    return load_library().infini_attn_status_string(int(status)).decode()


def _check(rc):
    if rc != OK:
        raise InfiniError(rc, status_string(rc))


def _stream_handle(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _one_device(first, *tensors, stream=None):
    """The library launches on the current CUDA device: every tensor (and the
    stream, if given) must be on the device of ``first``, which the call then
    makes current."""
    dev = first.device
    for t in tensors:
        if isinstance(t, torch.Tensor) and t.device != dev:
            raise ValueError(f"all tensors must be on {dev}; got one on {t.device}")
    if stream is not None and stream.device != dev:
        raise ValueError(f"the stream is on {stream.device}, the tensors on {dev}")
    return torch.cuda.device(dev)


def make_dims(B, H_q, H_kv, L, d_k, d_v, dtype):
    return Dims(B, H_q, H_kv, L, d_k, d_v, DTYPES[dtype] if isinstance(dtype, torch.dtype) else dtype)


def _dims_from(q, k, v):
    if q.dim() != 4 or k.dim() != 4 or v.dim() != 4:
        raise ValueError("q, k, v must be [B, H, L, d]")
    B, H_q, L, d_k = q.shape
    H_kv, d_v = k.shape[1], v.shape[-1]
    if tuple(k.shape) != (B, H_kv, L, d_k) or tuple(v.shape) != (B, H_kv, L, d_v):
        raise ValueError("k must be [B, H_kv, L, d_k] and v [B, H_kv, L, d_v]")
    if q.dtype not in DTYPES or k.dtype != q.dtype or v.dtype != q.dtype:
        raise ValueError("q, k, v must share one dtype, bfloat16 or float32")
    return make_dims(B, H_q, H_kv, L, d_k, d_v, q.dtype)


def _rule(rule):
    return RULES[rule] if isinstance(rule, str) else int(rule)


def workspace_bytes(dims, seg_len, rule):
    return load_library().infini_attn_workspace_bytes(ctypes.byref(dims), int(seg_len), _rule(rule))


def plan(dims, seg_len, rule):
    p = Plan()
    _check(load_library().infini_attn_plan(ctypes.byref(dims), int(seg_len), _rule(rule),
                                           ctypes.byref(p)))
    return {"path": PATHS.get(p.path, p.path), "launches": p.launches,
            "num_segments": p.num_segments, "workspace_bytes": p.workspace_bytes}


def init_state(B, H_kv, d_k, d_v, device=None, stream=None):
    """Allocate and zero (M, z) on the GPU through infini_attn_init_state."""
    device = device or torch.device("cuda", torch.cuda.current_device())
    M = torch.empty((B, H_kv, d_k, d_v), dtype=torch.float32, device=device)
    z = torch.empty((B, H_kv, d_k), dtype=torch.float32, device=device)
    _check(load_library().infini_attn_init_state(
        ctypes.c_void_p(M.data_ptr()), ctypes.c_void_p(z.data_ptr()), B, H_kv, d_k, d_v,
        _stream_handle(stream)))
    return M, z


def _dev(t, name, dtype=None, shape=None):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    return ctypes.c_void_p(t.data_ptr())


def forward(q, k, v, beta, M_in, z_in, seg_len, rule, out=None, M_out=None, z_out=None,
            workspace=None, stream=None):
    """infini_attn_forward on CUDA tensors; returns (out, M_out, z_out).

    Outputs are allocated when not given.  ``workspace`` is an optional uint8
    CUDA tensor of at least workspace_bytes(...) bytes; without it the library
    takes stream-ordered scratch itself.
    """
    lib = load_library()
    dims = _dims_from(q, k, v)
    B, H_q, L, H_kv, d_k, d_v = dims.B, dims.H_q, dims.L, dims.H_kv, dims.d_k, dims.d_v
    if out is None:
        out = torch.empty((B, H_q, L, d_v), dtype=q.dtype, device=q.device)
    if M_out is None:
        M_out = torch.empty((B, H_kv, d_k, d_v), dtype=torch.float32, device=q.device)
    if z_out is None:
        z_out = torch.empty((B, H_kv, d_k), dtype=torch.float32, device=q.device)
    args = [_dev(q, "q"), _dev(k, "k"), _dev(v, "v"),
            _dev(beta, "beta", torch.float32, (H_q,)),
            _dev(M_in, "M_in", torch.float32, (B, H_kv, d_k, d_v)),
            _dev(z_in, "z_in", torch.float32, (B, H_kv, d_k))]
    outs = [_dev(out, "out", q.dtype, (B, H_q, L, d_v)),
            _dev(M_out, "M_out", torch.float32, (B, H_kv, d_k, d_v)),
            _dev(z_out, "z_out", torch.float32, (B, H_kv, d_k))]
    if workspace is not None:
        ws_ptr, ws_n = _dev(workspace, "workspace", torch.uint8), workspace.numel()
    else:
        ws_ptr, ws_n = ctypes.c_void_p(0), 0
    with _one_device(q, k, v, beta, M_in, z_in, out, M_out, z_out, workspace, stream=stream):
        _check(lib.infini_attn_forward(*args, int(seg_len), _rule(rule), ctypes.byref(dims), *outs,
                                       ws_ptr, ws_n, _stream_handle(stream)))
    return out, M_out, z_out


def backward_workspace_bytes(dims, seg_len, rule):
    """infini_attn_backward_workspace_bytes (0 for unsupported shapes)."""
    return load_library().infini_attn_backward_workspace_bytes(ctypes.byref(dims), int(seg_len),
                                                               _rule(rule))


def backward(q, k, v, beta, M_in, z_in, seg_len, rule, dout, dM_out=None, dz_out=None,
             workspace=None, stream=None):
    """infini_attn_backward on CUDA tensors: the gradients of a loss with
    respect to the forward's inputs, given its gradients with respect to
    (out, M_out, z_out) (``dM_out`` / ``dz_out`` may be None for zero).
    Returns (dq, dk, dv, dbeta, dM_in, dz_in), all float32."""
    lib = load_library()
    dims = _dims_from(q, k, v)
    B, H_q, L, H_kv, d_k, d_v = dims.B, dims.H_q, dims.L, dims.H_kv, dims.d_k, dims.d_v
    f32 = dict(dtype=torch.float32, device=q.device)
    dq = torch.empty((B, H_q, L, d_k), **f32)
    dk = torch.empty((B, H_kv, L, d_k), **f32)
    dv = torch.empty((B, H_kv, L, d_v), **f32)
    dbeta = torch.empty((H_q,), **f32)
    dM_in = torch.empty((B, H_kv, d_k, d_v), **f32)
    dz_in = torch.empty((B, H_kv, d_k), **f32)
    args = [_dev(q, "q"), _dev(k, "k"), _dev(v, "v"),
            _dev(beta, "beta", torch.float32, (H_q,)),
            _dev(M_in, "M_in", torch.float32, (B, H_kv, d_k, d_v)),
            _dev(z_in, "z_in", torch.float32, (B, H_kv, d_k))]
    grads_in = [_dev(dout, "dout", q.dtype, (B, H_q, L, d_v)),
                _dev(dM_out, "dM_out", torch.float32, (B, H_kv, d_k, d_v))
                if dM_out is not None else ctypes.c_void_p(0),
                _dev(dz_out, "dz_out", torch.float32, (B, H_kv, d_k))
                if dz_out is not None else ctypes.c_void_p(0)]
    outs = [_dev(t, n) for t, n in ((dq, "dq"), (dk, "dk"), (dv, "dv"), (dbeta, "dbeta"),
                                     (dM_in, "dM_in"), (dz_in, "dz_in"))]
    if workspace is not None:
        ws_ptr, ws_n = _dev(workspace, "workspace", torch.uint8), workspace.numel()
    else:
        ws_ptr, ws_n = ctypes.c_void_p(0), 0
    with _one_device(q, k, v, beta, M_in, z_in, dout, dM_out, dz_out, workspace, stream=stream):
        _check(lib.infini_attn_backward(*args, int(seg_len), _rule(rule), ctypes.byref(dims),
                                        *grads_in, *outs, ws_ptr, ws_n, _stream_handle(stream)))
    return dq, dk, dv, dbeta, dM_in, dz_in


def state_update(k, v, M_in, z_in, seg_len, rule, M_out=None, z_out=None, workspace=None,
                 stream=None):
    """infini_attn_state_update on CUDA tensors: the state after the segments
    of k, v from (M_in, z_in); returns (M_out, z_out).  ``workspace``: an
    optional uint8 CUDA tensor of workspace_bytes(make_dims(B, H_kv, H_kv, L,
    d_k, d_v, dtype), seg_len, rule) bytes or more."""
    lib = load_library()
    if k.dim() != 4 or v.dim() != 4:
        raise ValueError("k and v must be [B, H_kv, L, d]")
    B, H_kv, L, d_k = k.shape
    d_v = v.shape[3]
    if tuple(v.shape[:3]) != (B, H_kv, L) or v.dtype != k.dtype:
        raise ValueError("v must match k in batch, heads, length and dtype")
    if k.dtype not in DTYPES:
        raise ValueError("k, v must be bfloat16 or float32")
    dims = make_dims(B, H_kv, H_kv, L, d_k, d_v, k.dtype)
    if M_out is None:
        M_out = torch.empty((B, H_kv, d_k, d_v), dtype=torch.float32, device=k.device)
    if z_out is None:
        z_out = torch.empty((B, H_kv, d_k), dtype=torch.float32, device=k.device)
    args = [_dev(k, "k"), _dev(v, "v"),
            _dev(M_in, "M_in", torch.float32, (B, H_kv, d_k, d_v)),
            _dev(z_in, "z_in", torch.float32, (B, H_kv, d_k))]
    outs = [_dev(M_out, "M_out", torch.float32, (B, H_kv, d_k, d_v)),
            _dev(z_out, "z_out", torch.float32, (B, H_kv, d_k))]
    if workspace is not None:
        ws_ptr, ws_n = _dev(workspace, "workspace", torch.uint8), workspace.numel()
    else:
        ws_ptr, ws_n = ctypes.c_void_p(0), 0
    with _one_device(k, v, M_in, z_in, M_out, z_out, workspace, stream=stream):
        _check(lib.infini_attn_state_update(*args, int(seg_len), _rule(rule), ctypes.byref(dims),
                                            *outs, ws_ptr, ws_n, _stream_handle(stream)))
    return M_out, z_out


def state_sum(M_base, z_base, parts, n_parts, M_out=None, z_out=None, stream=None):
    """infini_attn_state_sum: (M_base + the first ``n_parts`` packed states of
    ``parts`` (float32 CUDA tensor [n, B*H_kv*d_k*d_v + B*H_kv*d_k]), z_base
    likewise), summed in part order; returns (M_out, z_out)."""
    lib = load_library()
    B, H_kv, d_k, d_v = M_base.shape
    if M_out is None:
        M_out = torch.empty_like(M_base)
    if z_out is None:
        z_out = torch.empty_like(z_base)
    n_parts = int(n_parts)
    width = B * H_kv * d_k * (d_v + 1)
    if parts.dim() != 2 or parts.shape[1] != width or not 0 <= n_parts <= parts.shape[0]:
        raise ValueError(f"parts must be [n >= n_parts, {width}]")
    args = [_dev(M_base, "M_base", torch.float32, (B, H_kv, d_k, d_v)),
            _dev(z_base, "z_base", torch.float32, (B, H_kv, d_k)),
            _dev(parts, "parts", torch.float32) if n_parts > 0 else ctypes.c_void_p(0), n_parts,
            B, H_kv, d_k, d_v,
            _dev(M_out, "M_out", torch.float32, (B, H_kv, d_k, d_v)),
            _dev(z_out, "z_out", torch.float32, (B, H_kv, d_k))]
    with _one_device(M_base, z_base, parts, M_out, z_out, stream=stream):
        _check(lib.infini_attn_state_sum(*args, _stream_handle(stream)))
    return M_out, z_out


def rope_tables(n_pos, d, base=10000.0, device=None, stream=None):
    """infini_attn_rope_tables: float32 (cos, sin) [n_pos, d/2] on the GPU."""
    device = device or torch.device("cuda", torch.cuda.current_device())
    cos = torch.empty((n_pos, d // 2), dtype=torch.float32, device=device)
    sin = torch.empty((n_pos, d // 2), dtype=torch.float32, device=device)
    with _one_device(cos, sin, stream=stream):
        _check(load_library().infini_attn_rope_tables(
            ctypes.c_void_p(cos.data_ptr()), ctypes.c_void_p(sin.data_ptr()), int(n_pos), int(d),
            float(base), _stream_handle(stream)))
    return cos, sin


def qkv_project(x, w_qkv, bias, rope_cos, rope_sin, H_q, H_kv, d, q=None, k=None, v=None,
                stream=None):
    """infini_attn_qkv_project: x bf16 [B, L, d_model], w_qkv bf16
    [(H_q + 2 H_kv) d, d_model], bias float32 [(H_q + 2 H_kv) d] or None,
    rope_cos / rope_sin float32 [L, d/2] or None; returns bf16 (q, k, v) in
    the [B, H, L, d] layout of ``forward``."""
    lib = load_library()
    if x.dim() != 3:
        raise ValueError("x must be [B, L, d_model]")
    B, L, dm = x.shape
    n_out = (H_q + 2 * H_kv) * d
    if q is None:
        q = torch.empty((B, H_q, L, d), dtype=torch.bfloat16, device=x.device)
    if k is None:
        k = torch.empty((B, H_kv, L, d), dtype=torch.bfloat16, device=x.device)
    if v is None:
        v = torch.empty((B, H_kv, L, d), dtype=torch.bfloat16, device=x.device)
    if (rope_cos is None) != (rope_sin is None):
        raise ValueError("give both rotary tables or neither")
    rot = [ctypes.c_void_p(0), ctypes.c_void_p(0)]
    if rope_cos is not None:
        rot = [_dev(rope_cos, "rope_cos", torch.float32, (L, d // 2)),
               _dev(rope_sin, "rope_sin", torch.float32, (L, d // 2))]
    dims = make_dims(B, H_q, H_kv, L, d, d, torch.bfloat16)
    args = [_dev(x, "x", torch.bfloat16), _dev(w_qkv, "w_qkv", torch.bfloat16, (n_out, dm)),
            _dev(bias, "bias", torch.float32, (n_out,)) if bias is not None else ctypes.c_void_p(0),
            *rot, ctypes.byref(dims), int(dm),
            _dev(q, "q", torch.bfloat16, (B, H_q, L, d)), _dev(k, "k", torch.bfloat16, (B, H_kv, L, d)),
            _dev(v, "v", torch.bfloat16, (B, H_kv, L, d))]
    with _one_device(x, w_qkv, bias, rope_cos, rope_sin, q, k, v, stream=stream):
        _check(lib.infini_attn_qkv_project(*args, _stream_handle(stream)))
    return q, k, v


# The entry points below are called once per token or per layer, where the
# binding's own time counts: one check per tensor, plain integers as pointers,
# and no device switch when the tensors' device is current already.


def _arg(t, name, dtype, shape, dev):
    """Address of a contiguous tensor of exactly this type, shape and device;
    None for None."""
    if t is None:
        return None
    if t.dtype is not dtype or t.shape != shape or t.device != dev or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)} on {dev}, "
                         f"got {t.dtype} {tuple(t.shape)} on {t.device}")
    return t.data_ptr()


def _cuda_device(t, name):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    return t.device


def _workspace(t, dev):
    """(address, bytes) of an optional workspace tensor."""
    if t is None:
        return None, 0
    n = t.numel()
    return _arg(t, "workspace", torch.uint8, (n,), dev), n


@functools.lru_cache(maxsize=256)
def _strides(shape):
    """Strides of a contiguous tensor of this shape."""
    out, n = [], 1
    for s in reversed(shape):
        out.append(n)
        n *= max(s, 1)
    return tuple(reversed(out))


@functools.lru_cache(maxsize=256)
def _dims_ref(B, H_q, H_kv, L, d, dtype):
    """Reference to the struct of these sizes (calls only read it)."""
    if dtype not in DTYPES:
        raise ValueError("dtype must be bfloat16 or float32")
    return ctypes.byref(Dims(B, H_q, H_kv, L, d, d, DTYPES[dtype]))


def _empty(shape, dtype, dev, stream):
    """New memory for an output that ``stream`` writes: of that stream's pool.
    (empty_strided takes 1.6 us of the host's time, empty 2.5.)"""
    if stream is None:
        return torch.empty_strided(shape, _strides(shape), dtype=dtype, device=dev)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=dev)


def _output(t, name, dtype, shape, dev, stream):
    """(tensor, address) of an output: the caller's, checked, or new memory."""
    if t is None:
        t = _empty(shape, dtype, dev, stream)
        return t, t.data_ptr()
    return t, _arg(t, name, dtype, shape, dev)


def _like(t, stream):
    if stream is None:
        return torch.empty_like(t)
    with torch.cuda.stream(stream):
        return torch.empty_like(t)


# The current stream's handle without building a Stream object (0.1 us against
# 2.5 us); torch.cuda.current_stream where a torch build has no such call.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda index: torch.cuda.current_stream(index).cuda_stream)


def _call(fn, dev, stream, *args):
    """fn(*args, stream handle) with the tensors' device current."""
    index = dev.index
    if stream is None:
        handle = _raw_stream(index)
    elif stream.device != dev:
        raise ValueError(f"the stream is on {stream.device}, the tensors on {dev}")
    else:
        handle = stream.cuda_stream
    if torch.cuda.current_device() == index:
        rc = fn(*args, handle)
    else:
        with torch.cuda.device(dev):
            rc = fn(*args, handle)
    if rc != OK:
        _check(rc)


def block_norm(r, w_next, eps, o=None, gate=None, scale=None, w_post=None, r_out=None, h=None,
               keep_rstd=True, stream=None):
    """infini_attn_block_norm on CUDA tensors: r, o, gate [..., width] of one
    dtype (bfloat16 or float32), scale, w_post, w_next float32 [width].
    Returns (r_out, h, rstd_post, rstd_next): r_out is None without ``o``, h
    without ``w_next``, and the reciprocal norms (float32 [...], for
    block_norm_backward) without their weight or with ``keep_rstd=False``.
    ``r_out`` may be ``r`` itself."""
    dev, dt, shape = _cuda_device(r, "r"), r.dtype, r.shape
    if dt not in DTYPES or r.dim() < 1:
        raise ValueError("r must be [..., width], bfloat16 or float32")
    width, f32 = shape[-1], torch.float32
    vec, stat = (width,), shape[:-1]
    if not r.is_contiguous():
        raise ValueError("r must be contiguous")
    r_out_ptr = h_ptr = None
    if o is not None or r_out is not None:
        r_out, r_out_ptr = _output(r_out, "r_out", dt, shape, dev, stream)
    if w_next is not None or h is not None:
        h, h_ptr = _output(h, "h", dt, shape, dev, stream)
    rp = _empty(stat, f32, dev, stream) if keep_rstd and w_post is not None else None
    rn = _empty(stat, f32, dev, stream) if keep_rstd and w_next is not None else None
    _call(load_library().infini_attn_block_norm, dev, stream,
          _arg(r, "r", dt, shape, dev), _arg(o, "o", dt, shape, dev), _arg(gate, "gate", dt, shape, dev),
          _arg(scale, "scale", f32, vec, dev), _arg(w_post, "w_post", f32, vec, dev),
          _arg(w_next, "w_next", f32, vec, dev), eps, r.numel() // max(width, 1), width, DTYPES[dt],
          r_out_ptr, h_ptr, rp.data_ptr() if rp is not None else None, rn.data_ptr() if rn is not None else None)
    return r_out, h, rp, rn


class BlockNormGrads(NamedTuple):
    dr: Optional[torch.Tensor]
    do: Optional[torch.Tensor]
    dgate: Optional[torch.Tensor]
    dscale: Optional[torch.Tensor]
    dw_post: Optional[torch.Tensor]
    dw_next: Optional[torch.Tensor]


def block_norm_backward_workspace_bytes(rows, width):
    return load_library().infini_attn_block_norm_backward_workspace_bytes(int(rows), int(width))


def block_norm_backward(dr_out, dh, r_out, rstd_next, w_next, o=None, gate=None, scale=None,
                        w_post=None, rstd_post=None, workspace=None, stream=None):
    """infini_attn_block_norm_backward on CUDA tensors: the gradients of
    block_norm's inputs from those of its outputs (``dr_out`` may be None for
    zero; ``dh``, ``r_out`` and ``rstd_next`` are used with ``w_next`` only).
    Returns BlockNormGrads; a gradient whose input was absent is None, and
    without ``w_next`` dr is dr_out itself."""
    lead = dr_out if dr_out is not None else dh
    dev, dt, shape = _cuda_device(lead, "dr_out or dh"), lead.dtype, lead.shape
    if dt not in DTYPES or lead.dim() < 1 or not lead.is_contiguous():
        raise ValueError("gradients must be contiguous [..., width], bfloat16 or float32")
    width, f32 = shape[-1], torch.float32
    vec, stat = (width,), shape[:-1]
    if w_next is None:
        dh = r_out = rstd_next = None
    if w_post is None:
        rstd_post = None
    dr = _like(lead, stream) if w_next is not None else None
    d_o = _like(lead, stream) if o is not None else None
    dgate = _like(lead, stream) if gate is not None else None
    dscale, dw_post, dw_next = (_empty(vec, f32, dev, stream) if w is not None else None
                                for w in (scale, w_post, w_next))
    ws, ws_n = _workspace(workspace, dev)
    _call(load_library().infini_attn_block_norm_backward, dev, stream,
          _arg(dr_out, "dr_out", dt, shape, dev), _arg(dh, "dh", dt, shape, dev),
          _arg(r_out, "r_out", dt, shape, dev), _arg(o, "o", dt, shape, dev),
          _arg(gate, "gate", dt, shape, dev), _arg(scale, "scale", f32, vec, dev),
          _arg(w_post, "w_post", f32, vec, dev), _arg(w_next, "w_next", f32, vec, dev),
          _arg(rstd_post, "rstd_post", f32, stat, dev), _arg(rstd_next, "rstd_next", f32, stat, dev),
          lead.numel() // max(width, 1), width, DTYPES[dt],
          *(t.data_ptr() if t is not None else None for t in (dr, d_o, dgate, dscale, dw_post, dw_next)),
          ws, ws_n)
    return BlockNormGrads(dr if dr is not None else dr_out, d_o, dgate, dscale, dw_post, dw_next)


def _w4_shapes(N, K, group):
    blocks = -(-K // 128)
    return (N, blocks * 64), (N, blocks * 128 // group)


def w4_quantize(w, group=128, zeros=True, stream=None):
    """infini_attn_w4_quantize: w [N, K] (bfloat16 or float32 CUDA) to
    (packed uint8 [N, 64 ceil(K / 128)], scales bfloat16 and zeros uint8
    [N, ceil(K / 128) 128 / group]); zeros is None with ``zeros=False``."""
    dev = _cuda_device(w, "w")
    if w.dim() != 2 or w.dtype not in DTYPES or group not in (32, 64, 128):
        raise ValueError("w must be [N, K], bfloat16 or float32, and group 32, 64 or 128")
    N, K = w.shape
    ps, gs = _w4_shapes(N, K, group)
    packed = _empty(ps, torch.uint8, dev, stream)
    scales = _empty(gs, torch.bfloat16, dev, stream)
    z = _empty(gs, torch.uint8, dev, stream) if zeros else None
    _call(load_library().infini_attn_w4_quantize, dev, stream, _arg(w, "w", w.dtype, (N, K), dev), N, K,
          group, DTYPES[w.dtype], packed.data_ptr(), scales.data_ptr(), z.data_ptr() if zeros else None)
    return packed, scales, z


def w4_pack(codes, stream=None):
    """infini_attn_w4_pack: codes uint8 [N, K] (0..15) to packed uint8
    [N, 64 ceil(K / 128)]."""
    dev = _cuda_device(codes, "codes")
    if codes.dim() != 2:
        raise ValueError("codes must be [N, K]")
    N, K = codes.shape
    packed = _empty(_w4_shapes(N, K, 128)[0], torch.uint8, dev, stream)
    _call(load_library().infini_attn_w4_pack, dev, stream, _arg(codes, "codes", torch.uint8, (N, K), dev),
          N, K, packed.data_ptr())
    return packed


class LinearW4:
    """A linear layer with 4-bit weights (infini_attn_linear_w4 and
    infini_attn_qkv_project_w4): ``packed``, ``scales`` and ``zeros`` (or None)
    in the library's layout for K input channels, ``bias`` float32 [N] or None.
    The tensors are checked once, here; the object keeps them."""

    def __init__(self, packed, scales, zeros, K, bias=None):
        dev = self.device = _cuda_device(packed, "packed")
        if packed.dim() != 2 or scales.dim() != 2 or int(K) < 1:
            raise ValueError("packed must be [N, 64 ceil(K / 128)] and scales [N, groups]")
        self.N, self.K = packed.shape[0], int(K)
        padded = -(-self.K // 128) * 128
        groups = scales.shape[1]
        self.group = padded // groups if groups and padded % groups == 0 else 0
        if self.group not in (32, 64, 128):
            raise ValueError("scales must have ceil(K / 128) * 128 / group columns, group 32, 64 or 128")
        ps, gs = _w4_shapes(self.N, self.K, self.group)
        self.packed, self.scales, self.zeros, self.bias = packed, scales, zeros, bias
        self._weights = (_arg(packed, "packed", torch.uint8, ps, dev),
                         _arg(scales, "scales", torch.bfloat16, gs, dev),
                         _arg(zeros, "zeros", torch.uint8, gs, dev),
                         _arg(bias, "bias", torch.float32, (self.N,), dev))
        self._lib = load_library()

    @classmethod
    def from_weight(cls, w, group=128, zeros=True, bias=None, stream=None):
        """Quantise w [N, K]."""
        return cls(*w4_quantize(w, group, zeros, stream=stream), w.shape[1], bias=bias)

    def dequantize(self, dtype=torch.float32, stream=None):
        """The weights [N, K] as the layer uses them."""
        w = _empty((self.N, self.K), dtype, self.device, stream)
        _call(self._lib.infini_attn_w4_dequantize, self.device, stream, *self._weights[:3], self.N, self.K,
              self.group, DTYPES[dtype], w.data_ptr())
        return w

    def __call__(self, x, out=None, stream=None):
        """x [..., K], bfloat16 or float32, to [..., N] of the same type."""
        dt, shape = x.dtype, x.shape
        if dt not in DTYPES or not shape or shape[-1] != self.K:
            raise ValueError(f"x must be [..., {self.K}], bfloat16 or float32")
        ys = (*shape[:-1], self.N)
        y, y_ptr = _output(out, "out", dt, ys, self.device, stream)
        _call(self._lib.infini_attn_linear_w4, self.device, stream, _arg(x, "x", dt, shape, self.device),
              *self._weights, x.numel() // self.K, self.N, self.K, self.group, DTYPES[dt], y_ptr)
        return y

    def qkv(self, x, H_q, H_kv, d, rope_cos=None, rope_sin=None, positions=None, q=None, k=None, v=None,
            stream=None):
        """x [B, L, K] to the heads q [B, H_q, L, d], k, v [B, H_kv, L, d],
        queries and keys rotated by rows ``positions`` (int32 [B, L]; None:
        0 .. L - 1) of the float32 tables [n_pos, d / 2]."""
        dev, dt = self.device, x.dtype
        if dt not in DTYPES or x.dim() != 3 or x.shape[2] != self.K or (H_q + 2 * H_kv) * d != self.N:
            raise ValueError(f"x must be [B, L, {self.K}], bfloat16 or float32, and (H_q + 2 H_kv) d = {self.N}")
        if (rope_cos is None) != (rope_sin is None):
            raise ValueError("give both rotary tables or neither")
        B, L, _ = x.shape
        qs, ks = (B, H_q, L, d), (B, H_kv, L, d)
        q, q_ptr = _output(q, "q", dt, qs, dev, stream)
        k, k_ptr = _output(k, "k", dt, ks, dev, stream)
        v, v_ptr = _output(v, "v", dt, ks, dev, stream)
        n_pos = rope_cos.shape[0] if rope_cos is not None else 0
        rot = (n_pos, d // 2)
        _call(self._lib.infini_attn_qkv_project_w4, dev, stream, _arg(x, "x", dt, x.shape, dev),
              *self._weights, _arg(rope_cos, "rope_cos", torch.float32, rot, dev),
              _arg(rope_sin, "rope_sin", torch.float32, rot, dev), n_pos,
              _arg(positions, "positions", torch.int32, (B, L), dev), _dims_ref(B, H_q, H_kv, L, d, dt), self.K,
              self.group, q_ptr, k_ptr, v_ptr)
        return q, k, v


def decode_workspace_bytes(dims, seg_len, rule):
    return int(load_library().infini_attn_decode_workspace_bytes(ctypes.byref(dims), int(seg_len),
                                                                 _rule(rule)))


def decode_step(q_t, k_t, v_t, beta, k_buf, v_buf, pos, M, z, seg_len, rule, out=None,
                workspace=None, stream=None):
    """infini_attn_decode_step on CUDA tensors: q_t [B, H_q, d], k_t, v_t
    [B, H_kv, d], buffers [B, H_kv, seg_len, d]; (M, z) updated in place when
    pos == seg_len - 1.  Returns out [B, H_q, d]."""
    lib = load_library()
    if q_t.dim() != 3 or k_t.dim() != 3 or v_t.dim() != 3 or k_buf.dim() != 4:
        raise ValueError("q_t, k_t, v_t must be [B, heads, d] and the buffers [B, H_kv, S, d]")
    B, H_q, d = q_t.shape
    H_kv = k_t.shape[1]
    if q_t.dtype not in DTYPES:
        raise ValueError("dtype must be bfloat16 or float32")
    dims = make_dims(B, H_q, H_kv, 1, d, d, q_t.dtype)
    if out is None:
        out = torch.empty_like(q_t)
    buf = (B, H_kv, int(seg_len), d)
    args = [_dev(q_t, "q_t", q_t.dtype, (B, H_q, d)), _dev(k_t, "k_t", q_t.dtype, (B, H_kv, d)),
            _dev(v_t, "v_t", q_t.dtype, (B, H_kv, d)), _dev(beta, "beta", torch.float32, (H_q,)),
            _dev(k_buf, "k_buf", q_t.dtype, buf), _dev(v_buf, "v_buf", q_t.dtype, buf), int(pos),
            _dev(M, "M", torch.float32, (B, H_kv, d, d)), _dev(z, "z", torch.float32, (B, H_kv, d)),
            int(seg_len), _rule(rule), ctypes.byref(dims), _dev(out, "out", q_t.dtype, (B, H_q, d))]
    if workspace is not None:
        ws_ptr, ws_n = _dev(workspace, "workspace", torch.uint8), workspace.numel()
    else:
        ws_ptr, ws_n = ctypes.c_void_p(0), 0
    with _one_device(q_t, k_t, v_t, beta, k_buf, v_buf, M, z, out, workspace, stream=stream):
        _check(lib.infini_attn_decode_step(*args, ws_ptr, ws_n, _stream_handle(stream)))
    return out


class DecodeStream:
    """A stream decoded one token at a time: owns the segment buffers, the
    memory state and the position (marshalling around decode_step)."""

    def __init__(self, B, H_q, H_kv, d, seg_len, rule, dtype=torch.bfloat16, device=None,
                 M=None, z=None):
        device = torch.device("cuda") if device is None else device
        self.seg_len, self.rule, self.pos = int(seg_len), rule, 0
        self.k_buf = torch.zeros((B, H_kv, self.seg_len, d), dtype=dtype, device=device)
        self.v_buf = torch.zeros_like(self.k_buf)
        self.M = (torch.zeros((B, H_kv, d, d), dtype=torch.float32, device=device) if M is None
                  else M.clone())
        self.z = (torch.zeros((B, H_kv, d), dtype=torch.float32, device=device) if z is None
                  else z.clone())
        dims = make_dims(B, H_q, H_kv, 1, d, d, dtype)
        # zero-filled: the step's ticket counters start at 0
        self.workspace = torch.zeros(decode_workspace_bytes(dims, self.seg_len, rule),
                                     dtype=torch.uint8, device=device)

    def step(self, q_t, k_t, v_t, beta, out=None, stream=None):
        out = decode_step(q_t, k_t, v_t, beta, self.k_buf, self.v_buf, self.pos, self.M, self.z,
                          self.seg_len, self.rule, out=out, workspace=self.workspace, stream=stream)
        self.pos = (self.pos + 1) % self.seg_len
        return out

    def final_state(self, stream=None):
        """(M, z) after every token so far, counting a partly filled segment
        (the stream itself is left unchanged)."""
        if self.pos == 0:
            return self.M.clone(), self.z.clone()
        n = self.pos
        return state_update(self.k_buf[:, :, :n].contiguous(), self.v_buf[:, :, :n].contiguous(),
                            self.M, self.z, n, self.rule, stream=stream)


class CacheQ4:
    """A segment buffer in 4 bits (see infini_cache_q4_t): codes uint8
    [B, H_kv, S, d / 2] and scales bfloat16 [B, H_kv, S, d / 32, 2] of the keys
    and the values.  The tensors are checked once, here; the object keeps
    them."""

    def __init__(self, k_codes, k_scale, v_codes, v_scale):
        dev = self.device = _cuda_device(k_codes, "k_codes")
        if k_codes.dim() != 4:
            raise ValueError("k_codes must be [B, H_kv, S, d / 2]")
        B, H, S, half = k_codes.shape
        self.B, self.H_kv, self.seg_len, self.d = B, H, S, 2 * half
        if self.d not in (32, 64, 128) or S < 1:
            raise ValueError("the buffer's rows must hold 32, 64 or 128 channels")
        scale = (B, H, S, self.d // 32, 2)
        self.tensors = (k_codes, k_scale, v_codes, v_scale)
        self._ptrs = _CacheQ4Ptrs(_arg(k_codes, "k_codes", torch.uint8, k_codes.shape, dev),
                                  _arg(k_scale, "k_scale", torch.bfloat16, scale, dev),
                                  _arg(v_codes, "v_codes", torch.uint8, k_codes.shape, dev),
                                  _arg(v_scale, "v_scale", torch.bfloat16, scale, dev))
        self._ref = ctypes.byref(self._ptrs)
        self._lib = load_library()

    @classmethod
    def empty(cls, B, H_kv, seg_len, d, device=None):
        """A new buffer (zeros: every row reads as 0)."""
        device = device or torch.device("cuda", torch.cuda.current_device())
        codes = (B, H_kv, seg_len, d // 2)
        scale = (B, H_kv, seg_len, d // 32, 2)
        return cls(torch.zeros(codes, dtype=torch.uint8, device=device),
                   torch.zeros(scale, dtype=torch.bfloat16, device=device),
                   torch.zeros(codes, dtype=torch.uint8, device=device),
                   torch.zeros(scale, dtype=torch.bfloat16, device=device))

    def row(self, b):
        """Batch row b alone, as a view, for append, read and state_update (the decode
        step takes whole buffers)."""
        return CacheQ4(*(t[b:b + 1] for t in self.tensors))

    def _dims_ref(self, H_q, L, dtype):
        return _dims_ref(self.B, H_q, self.H_kv, L, self.d, dtype)

    def append(self, k, v, pos, stream=None):
        """infini_attn_cache_q4_append: k, v [B, H_kv, n, d] (bfloat16 or
        float32) into rows pos[b] .. pos[b] + n - 1, pos int32 [B]."""
        dev, dt, shape = self.device, k.dtype, k.shape
        if k.dim() != 4 or shape != (self.B, self.H_kv, shape[2], self.d):
            raise ValueError(f"k must be [{self.B}, {self.H_kv}, n, {self.d}]")
        _call(self._lib.infini_attn_cache_q4_append, dev, stream, _arg(k, "k", dt, shape, dev),
              _arg(v, "v", dt, shape, dev), _arg(pos, "pos", torch.int32, (self.B,), dev),
              self._dims_ref(self.H_kv, shape[2], dt), self.seg_len, self._ref)

    def read(self, n, dtype=torch.float32, k=None, v=None, stream=None):
        """infini_attn_cache_q4_read: the values of rows 0 .. n - 1, as
        (k, v) [B, H_kv, n, d]."""
        dev, shape = self.device, (self.B, self.H_kv, int(n), self.d)
        dims = self._dims_ref(self.H_kv, int(n), dtype)
        k, k_ptr = _output(k, "k", dtype, shape, dev, stream)
        v, v_ptr = _output(v, "v", dtype, shape, dev, stream)
        _call(self._lib.infini_attn_cache_q4_read, dev, stream, self._ref, dims, self.seg_len, k_ptr, v_ptr)
        return k, v

    def state_update(self, n, M_in, z_in, rule, dtype=torch.bfloat16, M_out=None, z_out=None,
                     workspace=None, stream=None):
        """infini_attn_state_update_q4: the memory after the first n rows as
        one segment; returns (M_out, z_out), which may be (M_in, z_in)."""
        dev, f32 = self.device, torch.float32
        ms, zs = (self.B, self.H_kv, self.d, self.d), (self.B, self.H_kv, self.d)
        dims = self._dims_ref(self.H_kv, int(n), dtype)
        M_out, M_ptr = _output(M_out, "M_out", f32, ms, dev, stream)
        z_out, z_ptr = _output(z_out, "z_out", f32, zs, dev, stream)
        ws, ws_n = _workspace(workspace, dev)
        _call(self._lib.infini_attn_state_update_q4, dev, stream, self._ref, _arg(M_in, "M_in", f32, ms, dev),
              _arg(z_in, "z_in", f32, zs, dev), _rule(rule), dims, self.seg_len,
              M_ptr, z_ptr, ws, ws_n)
        return M_out, z_out


def state_update_q4_workspace_bytes(B, H_kv, n, d, rule, dtype=torch.bfloat16):
    dims = make_dims(B, H_kv, H_kv, n, d, d, dtype)
    return load_library().infini_attn_state_update_q4_workspace_bytes(ctypes.byref(dims), _rule(rule))


def decode_q4_workspace_bytes(B, H_q, H_kv, seg_len, d):
    """infini_attn_decode_q4_workspace_bytes (0 for unsupported sizes)."""
    dims = make_dims(B, H_q, H_kv, 1, d, d, 0)
    return load_library().infini_attn_decode_q4_workspace_bytes(ctypes.byref(dims), int(seg_len))


def decode_step_q4(q_t, k_t, v_t, beta, cache, pos, M, z, out=None, workspace=None, stream=None):
    """infini_attn_decode_step_q4: q_t [B, H_q, d], k_t, v_t [B, H_kv, d]
    (bfloat16 or float32), ``cache`` a CacheQ4, pos int32 [B] (-1: idle), M, z
    the memory before the segment (read only).  ``workspace``: a uint8 tensor
    of decode_q4_workspace_bytes(...), zero-filled before its first step.
    Returns out [B, H_q, d]; idle rows of an ``out`` that is given keep what
    they hold, and are undefined in one that is not."""
    dev, dt, shape, f32 = cache.device, q_t.dtype, q_t.shape, torch.float32
    B, H, d = cache.B, cache.H_kv, cache.d
    if q_t.dim() != 3 or shape != (B, shape[1], d):
        raise ValueError(f"q_t must be [{B}, H_q, {d}]")
    tok = (B, H, d)
    dims = cache._dims_ref(shape[1], 1, dt)
    if out is None:
        out = _empty(shape, dt, dev, stream)
    ws, ws_n = _workspace(workspace, dev)
    _call(cache._lib.infini_attn_decode_step_q4, dev, stream, _arg(q_t, "q_t", dt, shape, dev),
          _arg(k_t, "k_t", dt, tok, dev), _arg(v_t, "v_t", dt, tok, dev),
          _arg(beta, "beta", f32, (shape[1],), dev), cache._ref, _arg(pos, "pos", torch.int32, (B,), dev),
          _arg(M, "M", f32, (B, H, d, d), dev), _arg(z, "z", f32, tok, dev), cache.seg_len, dims,
          _arg(out, "out", dt, shape, dev), ws, ws_n)
    return out


class DecodeStreamQ4:
    """DecodeStream with its segment buffer in 4 bits: one token per step for
    every stream, all at the same position (marshalling around decode_step_q4
    and CacheQ4.state_update)."""

    def __init__(self, B, H_q, H_kv, d, seg_len, rule, dtype=torch.bfloat16, device=None, M=None, z=None):
        device = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
        self.seg_len, self.rule, self.pos, self.dtype = int(seg_len), rule, 0, dtype
        self.cache = CacheQ4.empty(B, H_kv, self.seg_len, d, device)
        f32 = dict(dtype=torch.float32, device=device)
        self.M = torch.zeros((B, H_kv, d, d), **f32) if M is None else M.clone()
        self.z = torch.zeros((B, H_kv, d), **f32) if z is None else z.clone()
        self._pos = torch.zeros(B, dtype=torch.int32, device=device)
        # zero-filled: the step's ticket counters start at 0
        self.workspace = torch.zeros(decode_q4_workspace_bytes(B, H_q, H_kv, self.seg_len, d),
                                     dtype=torch.uint8, device=device)

    def step(self, q_t, k_t, v_t, beta, out=None):
        self._pos.fill_(self.pos)
        out = decode_step_q4(q_t, k_t, v_t, beta, self.cache, self._pos, self.M, self.z, out=out,
                             workspace=self.workspace)
        self.pos += 1
        if self.pos == self.seg_len:
            self.cache.state_update(self.seg_len, self.M, self.z, self.rule, self.dtype, self.M, self.z)
            self.pos = 0
        return out

    def final_state(self):
        """(M, z) after every token so far, counting a partly filled segment
        (the stream itself is left unchanged)."""
        if self.pos == 0:
            return self.M.clone(), self.z.clone()
        return self.cache.state_update(self.pos, self.M, self.z, self.rule, self.dtype)


def host_arena_bytes(dims, seg_len, rule):
    return load_library().infini_attn_host_arena_bytes(ctypes.byref(dims), int(seg_len), _rule(rule))


def _host(t, name, dtype=None, shape=None):
    if not isinstance(t, torch.Tensor) or t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous CPU tensor")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}")
    return ctypes.c_void_p(t.data_ptr())


def forward_host(q, k, v, beta, M_in, z_in, seg_len, rule, out, M_out, z_out, arena,
                 stream=None):
    """infini_attn_forward_host: host tensors in and out (pinned for async
    copies), device ``arena`` (uint8 CUDA tensor of host_arena_bytes(...))."""
    lib = load_library()
    dims = _dims_from(q, k, v)
    B, H_q, L, H_kv, d_k, d_v = dims.B, dims.H_q, dims.L, dims.H_kv, dims.d_k, dims.d_v
    args = [_host(q, "q"), _host(k, "k"), _host(v, "v"),
            _host(beta, "beta", torch.float32, (H_q,)),
            _host(M_in, "M_in", torch.float32, (B, H_kv, d_k, d_v)),
            _host(z_in, "z_in", torch.float32, (B, H_kv, d_k))]
    outs = [_host(out, "out", q.dtype, (B, H_q, L, d_v)),
            _host(M_out, "M_out", torch.float32, (B, H_kv, d_k, d_v)),
            _host(z_out, "z_out", torch.float32, (B, H_kv, d_k))]
    _check(lib.infini_attn_forward_host(*args, int(seg_len), _rule(rule), ctypes.byref(dims), *outs,
                                        _dev(arena, "arena", torch.uint8), arena.numel(),
                                        _stream_handle(stream)))
    return out, M_out, z_out


def sync_status(stream=None):
    """Wait for the stream; raise InfiniError(ERR_TIMEOUT) if a kernel gave up."""
    _check(load_library().infini_attn_sync_status(_stream_handle(stream)))


KERNEL_KINDS = ("state_scan", "attention")


def set_kernel_timing(enable):
    _check(load_library().infini_attn_set_kernel_timing(1 if enable else 0))


def kernel_times(reset=True):
    """{kind: (total ms, launches)} of the kernels timed since the last reset."""
    n = len(KERNEL_KINDS)
    ms = (ctypes.c_double * n)()
    cnt = (ctypes.c_int * n)()
    _check(load_library().infini_attn_kernel_times(ms, cnt, n, 1 if reset else 0))
    return {KERNEL_KINDS[i]: (ms[i], cnt[i]) for i in range(n)}


def noalloc_scratch_limit():
    return load_library().infini_attn_noalloc_scratch_limit()


def forward_noalloc(q, k, v, beta, M_in, z_in, seg_len, rule, out, M_out, z_out, stream=None):
    """infini_attn_forward_noalloc: the forward for callers that cannot allocate
    GPU memory while they run.  All outputs must be given (this wrapper
    allocates nothing either); scratch comes from the library's static array.
    """
    lib = load_library()
    dims = _dims_from(q, k, v)
    B, H_q, L, H_kv, d_k, d_v = dims.B, dims.H_q, dims.L, dims.H_kv, dims.d_k, dims.d_v
    args = [_dev(q, "q"), _dev(k, "k"), _dev(v, "v"),
            _dev(beta, "beta", torch.float32, (H_q,)),
            _dev(M_in, "M_in", torch.float32, (B, H_kv, d_k, d_v)),
            _dev(z_in, "z_in", torch.float32, (B, H_kv, d_k))]
    outs = [_dev(out, "out", q.dtype, (B, H_q, L, d_v)),
            _dev(M_out, "M_out", torch.float32, (B, H_kv, d_k, d_v)),
            _dev(z_out, "z_out", torch.float32, (B, H_kv, d_k))]
    with _one_device(q, k, v, beta, M_in, z_in, out, M_out, z_out, stream=stream):
        _check(lib.infini_attn_forward_noalloc(*args, int(seg_len), _rule(rule),
                                               ctypes.byref(dims), *outs, _stream_handle(stream)))
    return out, M_out, z_out


def selftest_approx(x, stream=None):
    """(poly 2^x, hardware 2^x, bf16 bits of |x|) computed on the GPU for the
    CUDA float32 tensor ``x`` by the kernel-side approximations."""
    x = x.contiguous()
    y_poly, y_mufu = torch.empty_like(x), torch.empty_like(x)
    bits = torch.empty(x.shape, dtype=torch.int32, device=x.device)
    _check(load_library().infini_attn_selftest_approx(
        _dev(x, "x", torch.float32), _dev(y_poly, "y_poly"), _dev(y_mufu, "y_mufu"),
        _dev(bits, "bits"), x.numel(), _stream_handle(stream)))
    return y_poly, y_mufu, bits


def selftest_timeout(stream=None):
    """Enqueue the bounded-wait failure-path self-check (one warp whose wait
    on a barrier nothing arrives at gives up after ~2 s and sets the device
    status word); a following sync_status raises InfiniError(ERR_TIMEOUT)."""
    _check(load_library().infini_attn_selftest_timeout(_stream_handle(stream)))
