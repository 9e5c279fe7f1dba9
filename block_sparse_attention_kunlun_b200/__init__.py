"""Block attention for NVIDIA B200 (sm_100a).

Python binding over the C ABI in ``include/ba.h`` (``libba.so`` in this
package directory, built by ``build.py``). The functions named like the C
entry points (``ba_fwd``, ``ba_bwd``, ...) marshal torch tensors into
pointers and call the library; every step of the computation runs in the
library's CUDA kernels. There is no CPU path: if the library is missing or
the device is not an sm_100 GPU, the calls raise.

Tensors: q, k, v, out, dout, dq, dk, dv are contiguous CUDA tensors of shape
``[total_tokens, heads, head_dim]`` (bfloat16 or float32); lse is float32
``[heads, total_tokens]``; seq_offsets is int32 ``[batch + 1]`` on the
device; skip is uint8 ``[batch]`` on the device or None.
"""
from __future__ import annotations

import ctypes
import os

import torch

__all__ = [
    "BAError", "ba_fwd", "ba_fwd_noalloc", "ba_bwd", "ba_fwd_workspace_size", "ba_bwd_workspace_size",
    "ba_swa_fwd", "ba_swa_bwd", "ba_swa_fwd_workspace_size", "ba_swa_bwd_workspace_size",
    "ba_rope_fwd", "ba_rope_bwd", "ba_rope_fwd_workspace_size", "ba_rope_bwd_workspace_size",
    "ba_device_status", "ba_selftest_wait_timeout", "ba_selftest_exp2", "ba_selftest_activation", "ba_set_profile_events", "ba_status_string", "ba_version",
    "block_attention_fwd", "block_attention_bwd", "sliding_window_attention_fwd", "sliding_window_attention_bwd",
    "rope_block_attention_fwd", "rope_block_attention_bwd",
    "ba_gdpa_workspace_size", "ba_gdpa_fwd", "ba_gdpa_bwd", "gdpa_fwd", "gdpa_bwd",
    "ba_gdpa_cross_workspace_size", "ba_gdpa_cross_fwd", "ba_gdpa_cross_bwd", "gdpa_cross_fwd", "gdpa_cross_bwd",
    "ba_mx_quantize", "ba_mx_fwd_workspace_size", "ba_mx_fwd", "mx_quantize", "mx_block_attention_fwd",
    "ba_mx_bwd_workspace_size", "ba_mx_bwd", "mx_block_attention_bwd",
    "HistoryCache", "ba_cache_write", "ba_cache_read", "ba_cache_summarize", "ba_cache_select", "ba_cache_fwd",
    "ba_cache_fwd_workspace_size", "cache_write", "cache_read", "cache_summarize", "cache_select",
    "cache_attention_fwd",
    "library_path",
]

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_HERE, "libba.so")

BA_OK, BA_ERR_INVALID_ARG, BA_ERR_UNSUPPORTED, BA_ERR_CUDA, BA_ERR_TIMEOUT = range(5)
BA_F32, BA_BF16 = 0, 1
BA_ACT_GELU, BA_ACT_SILU = 1, 2
_ACTS = {"gelu": BA_ACT_GELU, "silu": BA_ACT_SILU}
_DTYPES = {torch.float32: BA_F32, torch.bfloat16: BA_BF16}


class BAProblem(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("total_tokens", ctypes.c_int32),
                ("heads", ctypes.c_int32), ("head_dim", ctypes.c_int32), ("dtype", ctypes.c_int)]


class BARope(ctypes.Structure):
    _fields_ = [("cos", ctypes.c_void_p), ("sin", ctypes.c_void_p), ("rows", ctypes.c_int32),
                ("q_rot", ctypes.c_void_p), ("k_rot", ctypes.c_void_p)]


class BACache(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scales", ctypes.c_void_p),
                ("v_scales", ctypes.c_void_p), ("page_table", ctypes.c_void_p), ("status", ctypes.c_void_p),
                ("batch", ctypes.c_int32), ("max_pages", ctypes.c_int32), ("num_pages", ctypes.c_int32),
                ("page_size", ctypes.c_int32), ("kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32)]


class BAError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {ba_status_string(status)} ({status})")


_lib = None


def library_path() -> str:
    return _LIB_PATH


def _load():
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(_LIB_PATH):
        raise ImportError(f"{_LIB_PATH} is missing: build it with "
                          "`python -m block_sparse_attention_kunlun_b200.build`")
    lib = ctypes.CDLL(_LIB_PATH)
    P, i32 = ctypes.c_void_p, ctypes.c_int32
    prob = ctypes.POINTER(BAProblem)
    lib.ba_fwd_workspace_size.argtypes = [prob, i32, i32]
    lib.ba_fwd_workspace_size.restype = ctypes.c_size_t
    lib.ba_bwd_workspace_size.argtypes = [prob, i32, i32]
    lib.ba_bwd_workspace_size.restype = ctypes.c_size_t
    lib.ba_fwd.argtypes = [prob, P, P, P, P, i32, i32, P, P, P, P, ctypes.c_size_t, P]
    lib.ba_fwd.restype = ctypes.c_int
    lib.ba_bwd.argtypes = [prob, P, P, P, P, P, P, P, i32, i32, P, P, P, P, P, ctypes.c_size_t, P]
    lib.ba_bwd.restype = ctypes.c_int
    lib.ba_device_status.argtypes = [P, P]
    lib.ba_device_status.restype = ctypes.c_int
    lib.ba_status_string.argtypes = [ctypes.c_int]
    lib.ba_status_string.restype = ctypes.c_char_p
    lib.ba_fwd_noalloc.argtypes = [prob, P, P, P, P, i32, i32, P, P, P, P]
    lib.ba_fwd_noalloc.restype = ctypes.c_int
    lib.ba_set_profile_events.argtypes = [i32, P, P]
    lib.ba_set_profile_events.restype = ctypes.c_int
    lib.ba_version.argtypes = []
    lib.ba_version.restype = ctypes.c_int32
    lib.ba_selftest_wait_timeout.argtypes = [P, ctypes.c_size_t, i32, P]
    lib.ba_selftest_wait_timeout.restype = ctypes.c_int
    lib.ba_selftest_exp2.argtypes = [P, P, ctypes.c_int64, P]
    lib.ba_selftest_exp2.restype = ctypes.c_int
    lib.ba_selftest_activation.argtypes = [ctypes.c_int, P, P, P, ctypes.c_int64, P]
    lib.ba_selftest_activation.restype = ctypes.c_int
    lib.ba_swa_fwd_workspace_size.argtypes = [prob, i32]
    lib.ba_swa_fwd_workspace_size.restype = ctypes.c_size_t
    lib.ba_swa_bwd_workspace_size.argtypes = [prob, i32]
    lib.ba_swa_bwd_workspace_size.restype = ctypes.c_size_t
    lib.ba_swa_fwd.argtypes = [prob, P, P, P, P, i32, P, P, P, P, ctypes.c_size_t, P]
    lib.ba_swa_fwd.restype = ctypes.c_int
    lib.ba_swa_bwd.argtypes = [prob, P, P, P, P, P, P, P, i32, P, P, P, P, P, ctypes.c_size_t, P]
    lib.ba_swa_bwd.restype = ctypes.c_int
    lib.ba_gdpa_workspace_size.argtypes = [prob, i32, i32]
    lib.ba_gdpa_workspace_size.restype = ctypes.c_size_t
    lib.ba_gdpa_fwd.argtypes = [prob, ctypes.c_int, P, P, P, P, i32, i32, P, P, ctypes.c_size_t, P]
    lib.ba_gdpa_fwd.restype = ctypes.c_int
    lib.ba_gdpa_bwd.argtypes = [prob, ctypes.c_int, P, P, P, P, P, i32, i32, P, P, P, P, ctypes.c_size_t, P]
    lib.ba_gdpa_bwd.restype = ctypes.c_int
    lib.ba_gdpa_cross_workspace_size.argtypes = [prob, i32]
    lib.ba_gdpa_cross_workspace_size.restype = ctypes.c_size_t
    lib.ba_gdpa_cross_fwd.argtypes = [prob, i32, ctypes.c_int, P, P, P, P, P, P, P, ctypes.c_size_t, P]
    lib.ba_gdpa_cross_fwd.restype = ctypes.c_int
    lib.ba_gdpa_cross_bwd.argtypes = [prob, i32, ctypes.c_int, P, P, P, P, P, P, P, P, P, P, ctypes.c_size_t, P]
    lib.ba_gdpa_cross_bwd.restype = ctypes.c_int
    lib.ba_mx_quantize.argtypes = [P, ctypes.c_int64, i32, i32, P, P, P]
    lib.ba_mx_quantize.restype = ctypes.c_int
    lib.ba_mx_fwd_workspace_size.argtypes = [prob, i32, i32]
    lib.ba_mx_fwd_workspace_size.restype = ctypes.c_size_t
    lib.ba_mx_fwd.argtypes = [prob, P, P, P, P, i32, i32, P, P, P, P, ctypes.c_size_t, P]
    lib.ba_mx_fwd.restype = ctypes.c_int
    lib.ba_mx_bwd_workspace_size.argtypes = [prob, i32, i32]
    lib.ba_mx_bwd_workspace_size.restype = ctypes.c_size_t
    lib.ba_mx_bwd.argtypes = [prob, P, P, P, P, P, P, P, i32, i32, P, P, P, P, P, ctypes.c_size_t, P]
    lib.ba_mx_bwd.restype = ctypes.c_int
    cache = ctypes.POINTER(BACache)
    lib.ba_cache_write.argtypes = [cache, ctypes.c_int, P, P, P, P, i32, P]
    lib.ba_cache_write.restype = ctypes.c_int
    lib.ba_cache_read.argtypes = [cache, ctypes.c_int, P, P, i32, P, P, P]
    lib.ba_cache_read.restype = ctypes.c_int
    lib.ba_cache_summarize.argtypes = [cache, P, P, P, P]
    lib.ba_cache_summarize.restype = ctypes.c_int
    lib.ba_cache_select.argtypes = [cache, prob, P, P, P, P, P, i32, i32, i32, P, P]
    lib.ba_cache_select.restype = ctypes.c_int
    lib.ba_cache_fwd_workspace_size.argtypes = [cache, prob, i32, i32]
    lib.ba_cache_fwd_workspace_size.restype = ctypes.c_size_t
    lib.ba_cache_fwd.argtypes = [cache, prob, P, P, P, P, P, i32, P, i32, i32, P, P, P, ctypes.c_size_t, P]
    lib.ba_cache_fwd.restype = ctypes.c_int
    rope = ctypes.POINTER(BARope)
    lib.ba_rope_fwd_workspace_size.argtypes = [prob, i32, i32]
    lib.ba_rope_fwd_workspace_size.restype = ctypes.c_size_t
    lib.ba_rope_bwd_workspace_size.argtypes = [prob, i32, i32]
    lib.ba_rope_bwd_workspace_size.restype = ctypes.c_size_t
    lib.ba_rope_fwd.argtypes = [prob, rope, P, P, P, P, i32, i32, P, P, P, P, ctypes.c_size_t, P]
    lib.ba_rope_fwd.restype = ctypes.c_int
    lib.ba_rope_bwd.argtypes = [prob, rope, P, P, P, P, P, P, P, i32, i32, P, P, P, P, P, ctypes.c_size_t, P]
    lib.ba_rope_bwd.restype = ctypes.c_int
    _lib = lib
    return lib


def _ptr(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(stream):
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def make_problem(q: torch.Tensor, seq_offsets: torch.Tensor) -> BAProblem:
    if q.dim() != 3:
        raise ValueError("q must be [total_tokens, heads, head_dim]")
    if q.dtype not in _DTYPES:
        raise ValueError(f"unsupported dtype {q.dtype}")
    T, H, D = q.shape
    return BAProblem(int(seq_offsets.numel()) - 1, T, H, D, _DTYPES[q.dtype])


def ba_status_string(status: int) -> str:
    return _load().ba_status_string(int(status)).decode()


def ba_version() -> int:
    return int(_load().ba_version())


def ba_fwd_workspace_size(problem: BAProblem, block: int, window: int) -> int:
    return int(_load().ba_fwd_workspace_size(ctypes.byref(problem), int(block), int(window)))


def ba_bwd_workspace_size(problem: BAProblem, block: int, window: int) -> int:
    return int(_load().ba_bwd_workspace_size(ctypes.byref(problem), int(block), int(window)))


def ba_fwd(problem, q, k, v, seq_offsets, block, window, skip, out, lse, workspace,
           workspace_bytes=None, stream=None) -> int:
    """Direct call of the C entry point; returns its status code."""
    if workspace_bytes is None:
        workspace_bytes = workspace.numel() * workspace.element_size()
    return int(_load().ba_fwd(ctypes.byref(problem), _ptr(q), _ptr(k), _ptr(v), _ptr(seq_offsets),
                              int(block), int(window), _ptr(skip), _ptr(out), _ptr(lse),
                              _ptr(workspace), int(workspace_bytes), _stream(stream)))


def ba_fwd_noalloc(problem, q, k, v, seq_offsets, block, window, skip, out, lse, stream=None) -> int:
    """Direct call of the no-allocation forward (scratch inside the library)."""
    return int(_load().ba_fwd_noalloc(ctypes.byref(problem), _ptr(q), _ptr(k), _ptr(v), _ptr(seq_offsets),
                                      int(block), int(window), _ptr(skip), _ptr(out), _ptr(lse),
                                      _stream(stream)))


def ba_bwd(problem, q, k, v, out, lse, dout, seq_offsets, block, window, skip, dq, dk, dv,
           workspace, workspace_bytes=None, stream=None) -> int:
    """Direct call of the C entry point; returns its status code."""
    if workspace_bytes is None:
        workspace_bytes = workspace.numel() * workspace.element_size()
    return int(_load().ba_bwd(ctypes.byref(problem), _ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse),
                              _ptr(dout), _ptr(seq_offsets), int(block), int(window), _ptr(skip),
                              _ptr(dq), _ptr(dk), _ptr(dv), _ptr(workspace), int(workspace_bytes),
                              _stream(stream)))


def ba_swa_fwd_workspace_size(problem: BAProblem, window_tokens: int) -> int:
    return int(_load().ba_swa_fwd_workspace_size(ctypes.byref(problem), int(window_tokens)))


def ba_swa_bwd_workspace_size(problem: BAProblem, window_tokens: int) -> int:
    return int(_load().ba_swa_bwd_workspace_size(ctypes.byref(problem), int(window_tokens)))


def ba_swa_fwd(problem, q, k, v, seq_offsets, window_tokens, skip, out, lse, workspace,
               workspace_bytes=None, stream=None) -> int:
    """Direct call of the sliding-window forward; returns its status code."""
    if workspace_bytes is None:
        workspace_bytes = workspace.numel() * workspace.element_size()
    return int(_load().ba_swa_fwd(ctypes.byref(problem), _ptr(q), _ptr(k), _ptr(v), _ptr(seq_offsets),
                                  int(window_tokens), _ptr(skip), _ptr(out), _ptr(lse), _ptr(workspace),
                                  int(workspace_bytes), _stream(stream)))


def ba_swa_bwd(problem, q, k, v, out, lse, dout, seq_offsets, window_tokens, skip, dq, dk, dv,
               workspace, workspace_bytes=None, stream=None) -> int:
    """Direct call of the sliding-window backward; returns its status code."""
    if workspace_bytes is None:
        workspace_bytes = workspace.numel() * workspace.element_size()
    return int(_load().ba_swa_bwd(ctypes.byref(problem), _ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse),
                                  _ptr(dout), _ptr(seq_offsets), int(window_tokens), _ptr(skip),
                                  _ptr(dq), _ptr(dk), _ptr(dv), _ptr(workspace), int(workspace_bytes),
                                  _stream(stream)))


def _act(activation) -> int:
    if isinstance(activation, str):
        if activation not in _ACTS:
            raise ValueError(f"activation must be one of {sorted(_ACTS)}")
        return _ACTS[activation]
    return int(activation)


def ba_gdpa_workspace_size(problem: BAProblem, block: int, window: int) -> int:
    return int(_load().ba_gdpa_workspace_size(ctypes.byref(problem), int(block), int(window)))


def ba_gdpa_fwd(problem, activation, q, k, v, seq_offsets, block, window, out, workspace,
                workspace_bytes=None, stream=None) -> int:
    """Direct call of the generalized-attention forward; returns its status code."""
    if workspace_bytes is None:
        workspace_bytes = workspace.numel() * workspace.element_size()
    return int(_load().ba_gdpa_fwd(ctypes.byref(problem), _act(activation), _ptr(q), _ptr(k), _ptr(v),
                                   _ptr(seq_offsets), int(block), int(window), _ptr(out), _ptr(workspace),
                                   int(workspace_bytes), _stream(stream)))


def ba_gdpa_bwd(problem, activation, q, k, v, dout, seq_offsets, block, window, dq, dk, dv, workspace,
                workspace_bytes=None, stream=None) -> int:
    """Direct call of the generalized-attention backward; returns its status code."""
    if workspace_bytes is None:
        workspace_bytes = workspace.numel() * workspace.element_size()
    return int(_load().ba_gdpa_bwd(ctypes.byref(problem), _act(activation), _ptr(q), _ptr(k), _ptr(v),
                                   _ptr(dout), _ptr(seq_offsets), int(block), int(window), _ptr(dq), _ptr(dk),
                                   _ptr(dv), _ptr(workspace), int(workspace_bytes), _stream(stream)))


def gdpa_fwd(q, k, v, seq_offsets, block, window, activation="gelu", out=None, workspace=None, stream=None):
    """Generalized dot-product attention (activation in place of the softmax,
    block rule, no normalisation): allocates out (and a workspace) with torch
    and runs ba_gdpa_fwd."""
    _check_inputs(q, k, v, seq_offsets)
    prob = make_problem(q, seq_offsets)
    if out is None:
        out = _empty(q.shape, q.dtype, q.device, stream)
    if workspace is None:
        workspace = workspace_for(ba_gdpa_workspace_size(prob, block, window), q.device, stream)
    st = ba_gdpa_fwd(prob, activation, q, k, v, seq_offsets, block, window, out, workspace, stream=stream)
    if st != BA_OK:
        raise BAError(st, "ba_gdpa_fwd")
    return out


def gdpa_bwd(q, k, v, dout, seq_offsets, block, window, activation="gelu", dq=None, dk=None, dv=None,
             workspace=None, stream=None):
    """Gradients of gdpa_fwd: allocates dq/dk/dv (and a workspace) with torch and runs ba_gdpa_bwd."""
    _check_inputs(q, k, v, seq_offsets)
    prob = make_problem(q, seq_offsets)
    dq = _empty(q.shape, q.dtype, q.device, stream) if dq is None else dq
    dk = _empty(q.shape, q.dtype, q.device, stream) if dk is None else dk
    dv = _empty(q.shape, q.dtype, q.device, stream) if dv is None else dv
    if workspace is None:
        workspace = workspace_for(ba_gdpa_workspace_size(prob, block, window), q.device, stream)
    st = ba_gdpa_bwd(prob, activation, q, k, v, dout, seq_offsets, block, window, dq, dk, dv, workspace,
                     stream=stream)
    if st != BA_OK:
        raise BAError(st, "ba_gdpa_bwd")
    return dq, dk, dv


def ba_gdpa_cross_workspace_size(problem: BAProblem, kv_total_tokens: int) -> int:
    return int(_load().ba_gdpa_cross_workspace_size(ctypes.byref(problem), int(kv_total_tokens)))


def ba_gdpa_cross_fwd(problem, kv_total_tokens, activation, q, k, v, q_offsets, kv_offsets, out, workspace,
                      workspace_bytes=None, stream=None) -> int:
    """Direct call of the cross-attention GDPA forward; returns its status code."""
    if workspace_bytes is None:
        workspace_bytes = workspace.numel() * workspace.element_size()
    return int(_load().ba_gdpa_cross_fwd(ctypes.byref(problem), int(kv_total_tokens), _act(activation), _ptr(q),
                                         _ptr(k), _ptr(v), _ptr(q_offsets), _ptr(kv_offsets), _ptr(out),
                                         _ptr(workspace), int(workspace_bytes), _stream(stream)))


def ba_gdpa_cross_bwd(problem, kv_total_tokens, activation, q, k, v, dout, q_offsets, kv_offsets, dq, dk, dv,
                      workspace, workspace_bytes=None, stream=None) -> int:
    """Direct call of the cross-attention GDPA backward; returns its status code."""
    if workspace_bytes is None:
        workspace_bytes = workspace.numel() * workspace.element_size()
    return int(_load().ba_gdpa_cross_bwd(ctypes.byref(problem), int(kv_total_tokens), _act(activation), _ptr(q),
                                         _ptr(k), _ptr(v), _ptr(dout), _ptr(q_offsets), _ptr(kv_offsets),
                                         _ptr(dq), _ptr(dk), _ptr(dv), _ptr(workspace), int(workspace_bytes),
                                         _stream(stream)))


def _check_cross(q, k, v, q_offsets, kv_offsets):
    for name, t in (("q", q), ("k", k), ("v", v)):
        if not t.is_cuda or not t.is_contiguous() or t.dtype != q.dtype or t.dim() != 3:
            raise ValueError(f"{name} must be a contiguous CUDA tensor like q")
    if k.shape != v.shape or k.shape[1:] != q.shape[1:]:
        raise ValueError("k and v must be [kv_total_tokens, heads, head_dim] like q's heads and head_dim")
    for name, t in (("q_offsets", q_offsets), ("kv_offsets", kv_offsets)):
        if t.dtype != torch.int32 or not t.is_cuda:
            raise ValueError(f"{name} must be an int32 CUDA tensor")
    if q_offsets.numel() != kv_offsets.numel():
        raise ValueError("q_offsets and kv_offsets must describe the same examples")


def gdpa_cross_fwd(q, k, v, q_offsets, kv_offsets, activation="gelu", out=None, workspace=None, stream=None):
    """Cross-attention GDPA: example b's queries see every key of its own
    key/value set (no mask). Allocates out (and a workspace) with torch and
    runs ba_gdpa_cross_fwd."""
    _check_cross(q, k, v, q_offsets, kv_offsets)
    prob = make_problem(q, q_offsets)
    if out is None:
        out = _empty(q.shape, q.dtype, q.device, stream)
    if workspace is None:
        workspace = workspace_for(ba_gdpa_cross_workspace_size(prob, k.shape[0]), q.device, stream)
    st = ba_gdpa_cross_fwd(prob, k.shape[0], activation, q, k, v, q_offsets, kv_offsets, out, workspace,
                           stream=stream)
    if st != BA_OK:
        raise BAError(st, "ba_gdpa_cross_fwd")
    return out


def gdpa_cross_bwd(q, k, v, dout, q_offsets, kv_offsets, activation="gelu", dq=None, dk=None, dv=None,
                   workspace=None, stream=None):
    """Gradients of gdpa_cross_fwd (ba_gdpa_cross_bwd)."""
    _check_cross(q, k, v, q_offsets, kv_offsets)
    prob = make_problem(q, q_offsets)
    dq = _empty(q.shape, q.dtype, q.device, stream) if dq is None else dq
    dk = _empty(k.shape, k.dtype, k.device, stream) if dk is None else dk
    dv = _empty(v.shape, v.dtype, v.device, stream) if dv is None else dv
    if workspace is None:
        workspace = workspace_for(ba_gdpa_cross_workspace_size(prob, k.shape[0]), q.device, stream)
    st = ba_gdpa_cross_bwd(prob, k.shape[0], activation, q, k, v, dout, q_offsets, kv_offsets, dq, dk, dv,
                           workspace, stream=stream)
    if st != BA_OK:
        raise BAError(st, "ba_gdpa_cross_bwd")
    return dq, dk, dv


def ba_mx_quantize(x, elements, scales, stream=None) -> int:
    """Direct call of the MX (E4M3 / E8M0) quantisation of x [rows, heads, head_dim] bf16."""
    rows, heads, head_dim = x.shape
    return int(_load().ba_mx_quantize(_ptr(x), int(rows), int(heads), int(head_dim), _ptr(elements),
                                      _ptr(scales), _stream(stream)))


def mx_quantize(x, stream=None):
    """MX quantisation of a bf16 CUDA tensor [rows, heads, head_dim]: returns
    (elements uint8 [rows, heads, head_dim] holding E4M3 codes, scales uint8
    [rows, heads rounded up to 4, head_dim / 32] holding E8M0 codes)."""
    rows, heads, head_dim = x.shape
    elements = _empty(x.shape, torch.uint8, x.device, stream)
    shape = (rows, (heads + 3) // 4 * 4, head_dim // 32)
    scales = _empty(shape, torch.uint8, x.device, stream, make=torch.zeros)
    st = ba_mx_quantize(x, elements, scales, stream)
    if st != BA_OK:
        raise BAError(st, "ba_mx_quantize")
    return elements, scales


def ba_mx_fwd_workspace_size(problem: BAProblem, block: int, window: int) -> int:
    return int(_load().ba_mx_fwd_workspace_size(ctypes.byref(problem), int(block), int(window)))


def ba_mx_fwd(problem, q, k, v, seq_offsets, block, window, skip, out, lse, workspace, workspace_bytes=None,
              stream=None) -> int:
    """Direct call of the MXFP8-operand forward; returns its status code."""
    if workspace_bytes is None:
        workspace_bytes = workspace.numel() * workspace.element_size()
    return int(_load().ba_mx_fwd(ctypes.byref(problem), _ptr(q), _ptr(k), _ptr(v), _ptr(seq_offsets), int(block),
                                 int(window), _ptr(skip), _ptr(out), _ptr(lse), _ptr(workspace),
                                 int(workspace_bytes), _stream(stream)))


def mx_block_attention_fwd(q, k, v, seq_offsets, block, window, skip=None, out=None, lse=None, workspace=None,
                           stream=None):
    """Block attention with MXFP8 Q and K in the score product (ba_mx_fwd);
    allocates out/lse (and a workspace) with torch."""
    _check_inputs(q, k, v, seq_offsets)
    prob = make_problem(q, seq_offsets)
    if out is None:
        out = _empty(q.shape, q.dtype, q.device, stream)
    if lse is None:
        lse = _empty((q.shape[1], q.shape[0]), torch.float32, q.device, stream)
    if workspace is None:
        workspace = workspace_for(ba_mx_fwd_workspace_size(prob, block, window), q.device, stream)
    st = ba_mx_fwd(prob, q, k, v, seq_offsets, block, window, skip, out, lse, workspace, stream=stream)
    if st != BA_OK:
        raise BAError(st, "ba_mx_fwd")
    return out, lse


def ba_mx_bwd_workspace_size(problem: BAProblem, block: int, window: int) -> int:
    return int(_load().ba_mx_bwd_workspace_size(ctypes.byref(problem), int(block), int(window)))


def ba_mx_bwd(problem, q, k, v, out, lse, dout, seq_offsets, block, window, skip, dq, dk, dv,
              workspace, workspace_bytes=None, stream=None) -> int:
    """Direct call of the MXFP8-operand backward; returns its status code."""
    if workspace_bytes is None:
        workspace_bytes = workspace.numel() * workspace.element_size()
    return int(_load().ba_mx_bwd(ctypes.byref(problem), _ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse),
                                 _ptr(dout), _ptr(seq_offsets), int(block), int(window), _ptr(skip),
                                 _ptr(dq), _ptr(dk), _ptr(dv), _ptr(workspace), int(workspace_bytes),
                                 _stream(stream)))


def mx_block_attention_bwd(q, k, v, out, lse, dout, seq_offsets, block, window, skip=None,
                           dq=None, dk=None, dv=None, workspace=None, stream=None):
    """The backward of mx_block_attention_fwd (ba_mx_bwd); allocates dq/dk/dv
    (and a workspace) with torch."""
    _check_inputs(q, k, v, seq_offsets)
    prob = make_problem(q, seq_offsets)
    dq = _empty(q.shape, q.dtype, q.device, stream) if dq is None else dq
    dk = _empty(q.shape, q.dtype, q.device, stream) if dk is None else dk
    dv = _empty(q.shape, q.dtype, q.device, stream) if dv is None else dv
    if workspace is None:
        workspace = workspace_for(ba_mx_bwd_workspace_size(prob, block, window), q.device, stream)
    st = ba_mx_bwd(prob, q, k, v, out, lse, dout, seq_offsets, block, window, skip, dq, dk, dv, workspace,
                   stream=stream)
    if st != BA_OK:
        raise BAError(st, "ba_mx_bwd")
    return dq, dk, dv


def make_rope(cos, sin, q_rot=None, k_rot=None) -> BARope:
    """Rotary tables (float32 CUDA tensors [rows, head_dim / 2]) as the C
    struct, with optional caller buffers for the rotated q and k."""
    for name, t in (("cos", cos), ("sin", sin)):
        if not isinstance(t, int) and (t.dtype != torch.float32 or t.dim() != 2 or not t.is_contiguous()):
            raise ValueError(f"{name} must be a contiguous float32 [rows, head_dim / 2] tensor")
    rows = cos.shape[0] if not isinstance(cos, int) else 0
    return BARope(_ptr(cos), _ptr(sin), int(rows), _ptr(q_rot), _ptr(k_rot))


def ba_rope_fwd_workspace_size(problem: BAProblem, block: int, window: int) -> int:
    return int(_load().ba_rope_fwd_workspace_size(ctypes.byref(problem), int(block), int(window)))


def ba_rope_bwd_workspace_size(problem: BAProblem, block: int, window: int) -> int:
    return int(_load().ba_rope_bwd_workspace_size(ctypes.byref(problem), int(block), int(window)))


def ba_rope_fwd(problem, rope, q, k, v, seq_offsets, block, window, skip, out, lse, workspace,
                workspace_bytes=None, stream=None) -> int:
    """Direct call of the rotary forward (rope: BARope or None); returns its status code."""
    if workspace_bytes is None:
        workspace_bytes = workspace.numel() * workspace.element_size()
    return int(_load().ba_rope_fwd(ctypes.byref(problem), ctypes.byref(rope) if rope is not None else None,
                                   _ptr(q), _ptr(k), _ptr(v), _ptr(seq_offsets), int(block), int(window),
                                   _ptr(skip), _ptr(out), _ptr(lse), _ptr(workspace), int(workspace_bytes),
                                   _stream(stream)))


def ba_rope_bwd(problem, rope, q, k, v, out, lse, dout, seq_offsets, block, window, skip, dq, dk, dv,
                workspace, workspace_bytes=None, stream=None) -> int:
    """Direct call of the rotary backward; returns its status code."""
    if workspace_bytes is None:
        workspace_bytes = workspace.numel() * workspace.element_size()
    return int(_load().ba_rope_bwd(ctypes.byref(problem), ctypes.byref(rope) if rope is not None else None,
                                   _ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), _ptr(dout),
                                   _ptr(seq_offsets), int(block), int(window), _ptr(skip), _ptr(dq), _ptr(dk),
                                   _ptr(dv), _ptr(workspace), int(workspace_bytes), _stream(stream)))


def ba_set_profile_events(which: int, start=None, stop=None) -> int:
    """Record torch.cuda.Event ``start``/``stop`` around one kernel of every
    later call from this thread: 0 the forward attention kernel, 1 the
    backward dQ kernel, 2 the backward dK/dV kernel.
    The events must already exist on the device (torch creates an event on
    its first ``record``)."""
    s = start.cuda_event if start is not None else None
    e = stop.cuda_event if stop is not None else None
    if (start is not None and not s) or (stop is not None and not e):
        raise ValueError("record each event once before handing it to the library")
    return int(_load().ba_set_profile_events(int(which), s, e))


def ba_selftest_wait_timeout(workspace, limit_us: int, workspace_bytes=None, stream=None) -> int:
    """Launch the bounded-wait self-test (a wait that must time out); returns its status code."""
    if workspace_bytes is None:
        workspace_bytes = workspace.numel() * workspace.element_size()
    return int(_load().ba_selftest_wait_timeout(_ptr(workspace), int(workspace_bytes), int(limit_us),
                                                _stream(stream)))


def ba_selftest_exp2(x, y, stream=None) -> int:
    """y = the kernels' FMA-pipe 2^x for float32 CUDA tensors x, y of equal size."""
    if x.dtype != torch.float32 or y.dtype != torch.float32 or x.numel() != y.numel():
        raise ValueError("x and y must be float32 tensors of equal size")
    return int(_load().ba_selftest_exp2(_ptr(x), _ptr(y), int(x.numel()), _stream(stream)))


def ba_selftest_activation(act, x, y, dy, stream=None) -> int:
    """y = act(x), dy = act'(x) through the generalized attention's device
    functions (act: BA_ACT_GELU or BA_ACT_SILU), float32 CUDA tensors of equal size."""
    if any(t.dtype != torch.float32 or t.numel() != x.numel() for t in (x, y, dy)):
        raise ValueError("x, y and dy must be float32 tensors of equal size")
    return int(_load().ba_selftest_activation(int(act), _ptr(x), _ptr(y), _ptr(dy), int(x.numel()),
                                              _stream(stream)))


def ba_device_status(workspace, stream=None) -> int:
    return int(_load().ba_device_status(_ptr(workspace), _stream(stream)))


def _check_inputs(q, k, v, seq_offsets):
    for name, t in (("q", q), ("k", k), ("v", v)):
        if not t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous CUDA tensor")
        if t.shape != q.shape or t.dtype != q.dtype:
            raise ValueError(f"{name} must match q in shape and dtype")
    if seq_offsets.dtype != torch.int32 or not seq_offsets.is_cuda:
        raise ValueError("seq_offsets must be an int32 CUDA tensor")


def _launch_stream(stream, device):
    """The stream argument of a call as torch's stream on `device`."""
    if isinstance(stream, torch.cuda.Stream):
        return stream
    raw = _stream(stream)
    # (0 and 1 are both CUDA's default stream)
    return torch.cuda.ExternalStream(raw, device=device) if raw > 1 else torch.cuda.default_stream(device)


def _empty(shape, dtype, device, stream, returned=True, make=torch.empty):
    """An uninitialised (or make's) tensor for a call that launches on `stream` (None: the current one). Torch reuses a
    freed block in the order of the stream it was allocated on, so it is allocated on the call's; a tensor that
    is returned stays out of reuse until the work of the caller's stream at its end is done, too."""
    if stream is None:
        return make(shape, dtype=dtype, device=device)
    launch = _launch_stream(stream, device)
    caller = torch.cuda.current_stream(device)
    with torch.cuda.stream(launch):
        t = make(shape, dtype=dtype, device=device)
    if returned and launch != caller:
        t.record_stream(caller)
    return t


def workspace_for(nbytes: int, device, stream=None) -> torch.Tensor:
    """A workspace for calls on `stream` (None: the current one)."""
    # torch's caching allocator returns 512-byte-aligned blocks
    return _empty(max(int(nbytes), 256), torch.uint8, device, stream, returned=False)


def block_attention_fwd(q, k, v, seq_offsets, block, window, skip=None, out=None, lse=None,
                        workspace=None, stream=None):
    """Allocates out/lse (and a workspace) with torch and runs ba_fwd."""
    _check_inputs(q, k, v, seq_offsets)
    prob = make_problem(q, seq_offsets)
    if out is None:
        out = _empty(q.shape, q.dtype, q.device, stream)
    if lse is None:
        lse = _empty((q.shape[1], q.shape[0]), torch.float32, q.device, stream)
    if workspace is None:
        workspace = workspace_for(ba_fwd_workspace_size(prob, block, window), q.device, stream)
    st = ba_fwd(prob, q, k, v, seq_offsets, block, window, skip, out, lse, workspace, stream=stream)
    if st != BA_OK:
        raise BAError(st, "ba_fwd")
    return out, lse


def block_attention_bwd(q, k, v, out, lse, dout, seq_offsets, block, window, skip=None,
                        dq=None, dk=None, dv=None, workspace=None, stream=None):
    """Allocates dq/dk/dv (and a workspace) with torch and runs ba_bwd."""
    _check_inputs(q, k, v, seq_offsets)
    prob = make_problem(q, seq_offsets)
    dq = _empty(q.shape, q.dtype, q.device, stream) if dq is None else dq
    dk = _empty(q.shape, q.dtype, q.device, stream) if dk is None else dk
    dv = _empty(q.shape, q.dtype, q.device, stream) if dv is None else dv
    if workspace is None:
        workspace = workspace_for(ba_bwd_workspace_size(prob, block, window), q.device, stream)
    st = ba_bwd(prob, q, k, v, out, lse, dout, seq_offsets, block, window, skip, dq, dk, dv,
                workspace, stream=stream)
    if st != BA_OK:
        raise BAError(st, "ba_bwd")
    return dq, dk, dv


def sliding_window_attention_fwd(q, k, v, seq_offsets, window_tokens, skip=None, out=None, lse=None,
                                 workspace=None, stream=None):
    """Allocates out/lse (and a workspace) with torch and runs ba_swa_fwd:
    query i sees keys i - window_tokens < j <= i of its example."""
    _check_inputs(q, k, v, seq_offsets)
    prob = make_problem(q, seq_offsets)
    if out is None:
        out = _empty(q.shape, q.dtype, q.device, stream)
    if lse is None:
        lse = _empty((q.shape[1], q.shape[0]), torch.float32, q.device, stream)
    if workspace is None:
        workspace = workspace_for(ba_swa_fwd_workspace_size(prob, window_tokens), q.device, stream)
    st = ba_swa_fwd(prob, q, k, v, seq_offsets, window_tokens, skip, out, lse, workspace, stream=stream)
    if st != BA_OK:
        raise BAError(st, "ba_swa_fwd")
    return out, lse


def sliding_window_attention_bwd(q, k, v, out, lse, dout, seq_offsets, window_tokens, skip=None,
                                 dq=None, dk=None, dv=None, workspace=None, stream=None):
    """Allocates dq/dk/dv (and a workspace) with torch and runs ba_swa_bwd."""
    _check_inputs(q, k, v, seq_offsets)
    prob = make_problem(q, seq_offsets)
    dq = _empty(q.shape, q.dtype, q.device, stream) if dq is None else dq
    dk = _empty(q.shape, q.dtype, q.device, stream) if dk is None else dk
    dv = _empty(q.shape, q.dtype, q.device, stream) if dv is None else dv
    if workspace is None:
        workspace = workspace_for(ba_swa_bwd_workspace_size(prob, window_tokens), q.device, stream)
    st = ba_swa_bwd(prob, q, k, v, out, lse, dout, seq_offsets, window_tokens, skip, dq, dk, dv,
                    workspace, stream=stream)
    if st != BA_OK:
        raise BAError(st, "ba_swa_bwd")
    return dq, dk, dv


def _check_tables(cos, sin, q):
    for name, t in (("cos", cos), ("sin", sin)):
        if not t.is_cuda or t.dtype != torch.float32 or t.dim() != 2 or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous float32 CUDA tensor [rows, head_dim / 2]")
        if t.shape[1] != q.shape[2] // 2 or t.shape != cos.shape:
            raise ValueError("cos and sin must both be [rows, head_dim / 2]")


def _check_rotated(q_rot, k_rot, q):
    if (q_rot is None) != (k_rot is None):
        raise ValueError("pass both q_rot and k_rot, or neither")
    for name, t in (("q_rot", q_rot), ("k_rot", k_rot)):
        if t is not None and (not t.is_cuda or not t.is_contiguous() or t.shape != q.shape or t.dtype != q.dtype):
            raise ValueError(f"{name} must be a contiguous CUDA tensor like q")


def rope_block_attention_fwd(q, k, v, seq_offsets, block, window, cos, sin, skip=None, out=None, lse=None,
                             workspace=None, q_rot=None, k_rot=None, stream=None):
    """Rotary embedding on q and k (tables cos, sin [rows, head_dim / 2];
    rows must cover the longest example), then block attention: ba_rope_fwd.
    Allocates out/lse (and a workspace) with torch. q_rot / k_rot: buffers
    like q that receive the rotated q and k, to hand to the backward."""
    _check_inputs(q, k, v, seq_offsets)
    _check_tables(cos, sin, q)
    _check_rotated(q_rot, k_rot, q)
    prob = make_problem(q, seq_offsets)
    if out is None:
        out = _empty(q.shape, q.dtype, q.device, stream)
    if lse is None:
        lse = _empty((q.shape[1], q.shape[0]), torch.float32, q.device, stream)
    if workspace is None:
        need = (ba_fwd_workspace_size if q_rot is not None else ba_rope_fwd_workspace_size)(prob, block, window)
        workspace = workspace_for(need, q.device, stream)
    st = ba_rope_fwd(prob, make_rope(cos, sin, q_rot, k_rot), q, k, v, seq_offsets, block, window, skip, out,
                     lse, workspace, stream=stream)
    if st != BA_OK:
        raise BAError(st, "ba_rope_fwd")
    return out, lse


def rope_block_attention_bwd(q, k, v, out, lse, dout, seq_offsets, block, window, cos, sin, skip=None,
                             dq=None, dk=None, dv=None, workspace=None, q_rot=None, k_rot=None, stream=None):
    """Gradients of rope_block_attention_fwd with respect to the unrotated q,
    k and v: ba_rope_bwd. Allocates dq/dk/dv (and a workspace) with torch.
    q_rot / k_rot: the forward's rotated copies (then no rotation pass runs)."""
    _check_inputs(q, k, v, seq_offsets)
    _check_tables(cos, sin, q)
    _check_rotated(q_rot, k_rot, q)
    prob = make_problem(q, seq_offsets)
    dq = _empty(q.shape, q.dtype, q.device, stream) if dq is None else dq
    dk = _empty(q.shape, q.dtype, q.device, stream) if dk is None else dk
    dv = _empty(q.shape, q.dtype, q.device, stream) if dv is None else dv
    if workspace is None:
        need = (ba_bwd_workspace_size if q_rot is not None else ba_rope_bwd_workspace_size)(prob, block, window)
        workspace = workspace_for(need, q.device, stream)
    st = ba_rope_bwd(prob, make_rope(cos, sin, q_rot, k_rot), q, k, v, out, lse, dout, seq_offsets, block,
                     window, skip, dq, dk, dv, workspace, stream=stream)
    if st != BA_OK:
        raise BAError(st, "ba_rope_bwd")
    return dq, dk, dv


# ------------------------------------------------------- history cache ---

class HistoryCache:
    """A paged cache of keys and values in MXFP8 (ba_cache in include/ba.h).

    k, v: uint8 [num_pages, kv_heads, page_size, head_dim] (E4M3 codes);
    k_scales, v_scales: uint8 [num_pages, kv_heads, page_size, head_dim / 32]
    (E8M0 codes); page_table: int32 [batch, max_pages]; status: int32 CUDA
    tensor of one word, zeroed here when not given. The tensors are kept, not
    copied, and the calls read their addresses as they were: the caller changes
    page_table in place as histories grow, and makes another HistoryCache on the
    same pools for a wider one (attributes cannot be assigned to).
    """

    __slots__ = ("k", "v", "k_scales", "v_scales", "page_table", "status", "struct", "batch", "device", "_ref",
                 "_index", "_row", "_words")

    def __init__(self, k, v, k_scales, v_scales, page_table, status=None):
        if k.dim() != 4:
            raise ValueError("k must be [num_pages, kv_heads, page_size, head_dim]")
        num_pages, kv_heads, page_size, head_dim = k.shape
        if page_table.dim() != 2 or page_table.dtype != torch.int32:
            raise ValueError("page_table must be int32 [batch, max_pages]")
        if status is None:
            status = torch.zeros(1, dtype=torch.int32, device=k.device)
        for name, t, shape in (("k", k, k.shape), ("v", v, k.shape),
                               ("k_scales", k_scales, (*k.shape[:3], head_dim // 32)),
                               ("v_scales", v_scales, (*k.shape[:3], head_dim // 32))):
            if t.dtype != torch.uint8 or tuple(t.shape) != tuple(shape):
                raise ValueError(f"{name} must be uint8 {list(shape)}")
        if status.dtype != torch.int32 or status.numel() < 1:
            raise ValueError("status must be an int32 tensor")
        for name, t in (("k", k), ("v", v), ("k_scales", k_scales), ("v_scales", v_scales),
                        ("page_table", page_table), ("status", status)):
            if not t.is_cuda or not t.is_contiguous() or t.device != k.device:
                raise ValueError(f"{name} must be a contiguous CUDA tensor on k's device")
        struct = BACache(k.data_ptr(), v.data_ptr(), k_scales.data_ptr(), v_scales.data_ptr(),
                         page_table.data_ptr(), status.data_ptr(), page_table.shape[0], page_table.shape[1],
                         num_pages, page_size, kv_heads, head_dim)
        for name, x in (("k", k), ("v", v), ("k_scales", k_scales), ("v_scales", v_scales),
                        ("page_table", page_table), ("status", status), ("struct", struct),
                        ("batch", page_table.shape[0]), ("device", k.device), ("_ref", ctypes.byref(struct)),
                        ("_index", k.get_device()), ("_row", (kv_heads, head_dim)),
                        ("_words", (page_table.shape[1] + 31) // 32)):
            object.__setattr__(self, name, x)

    def __setattr__(self, name, value):
        raise AttributeError(f"{name} is the cache's for good: change its contents, or make another HistoryCache")

    def __delattr__(self, name):
        self.__setattr__(name, None)

    def __reduce__(self):
        return HistoryCache, (self.k, self.v, self.k_scales, self.v_scales, self.page_table, self.status)

    @classmethod
    def empty(cls, num_pages, page_size, kv_heads, head_dim, page_table):
        """A cache of zeroed pages on page_table's device."""
        shape = (num_pages, kv_heads, page_size, head_dim)
        k, v = (torch.zeros(shape, dtype=torch.uint8, device=page_table.device) for _ in "kv")
        ks, vs = (torch.zeros((*shape[:3], head_dim // 32), dtype=torch.uint8, device=page_table.device) for _ in "kv")
        return cls(k, v, ks, vs, page_table)


def _cache_ref(cache):
    return cache._ref if isinstance(cache, HistoryCache) else ctypes.byref(cache)


def ba_cache_write(cache, dtype, k, v, row_offsets, starts, total_rows, stream=None) -> int:
    """Direct call of the C entry point (cache: HistoryCache or BACache); returns its status code."""
    return int(_load().ba_cache_write(_cache_ref(cache), int(dtype), _ptr(k), _ptr(v), _ptr(row_offsets),
                                      _ptr(starts), int(total_rows), _stream(stream)))


def ba_cache_read(cache, dtype, row_offsets, starts, total_rows, k, v, stream=None) -> int:
    """Direct call of the C entry point; returns its status code."""
    return int(_load().ba_cache_read(_cache_ref(cache), int(dtype), _ptr(row_offsets), _ptr(starts),
                                     int(total_rows), _ptr(k), _ptr(v), _stream(stream)))


def ba_cache_summarize(cache, starts, ends, summaries, stream=None) -> int:
    """Direct call of the C entry point; returns its status code."""
    return int(_load().ba_cache_summarize(_cache_ref(cache), _ptr(starts), _ptr(ends), _ptr(summaries),
                                          _stream(stream)))


def ba_cache_select(cache, problem, q, q_offsets, lens, positions, summaries, block, window, topk, page_mask,
                    stream=None) -> int:
    """Direct call of the C entry point; returns its status code."""
    return int(_load().ba_cache_select(_cache_ref(cache), ctypes.byref(problem), _ptr(q), _ptr(q_offsets),
                                       _ptr(lens), _ptr(positions), _ptr(summaries), int(block), int(window),
                                       int(topk), _ptr(page_mask), _stream(stream)))


def ba_cache_fwd_workspace_size(cache, problem: BAProblem, block: int, window: int) -> int:
    return int(_load().ba_cache_fwd_workspace_size(_cache_ref(cache), ctypes.byref(problem), int(block), int(window)))


def ba_cache_fwd(cache, problem, q, q_offsets, lens, positions, tree_mask, tree_words, page_mask, block, window, out,
                 lse, workspace, workspace_bytes=None, stream=None) -> int:
    """Direct call of the C entry point; returns its status code."""
    if workspace_bytes is None:
        workspace_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    return int(_load().ba_cache_fwd(_cache_ref(cache), ctypes.byref(problem), _ptr(q), _ptr(q_offsets), _ptr(lens),
                                    _ptr(positions), _ptr(tree_mask), int(tree_words), _ptr(page_mask), int(block),
                                    int(window), _ptr(out), _ptr(lse), _ptr(workspace), int(workspace_bytes),
                                    _stream(stream)))


def _fits(cache, t, dtype, shape) -> bool:
    """A contiguous tensor of this type and shape on the cache's device."""
    return t.dtype is dtype and t.shape == shape and t.get_device() == cache._index and t.is_contiguous()


def _refuse(cache, named):
    """The ValueError for the first of (name, tensor, dtype, shape) that does not fit."""
    for name, t, dtype, shape in named:
        if not _fits(cache, t, dtype, shape):
            raise ValueError(f"{name} must be a contiguous {dtype} tensor {list(shape)} on {cache.device}")
    raise ValueError(f"the cache is on {cache.device}: make it the current device")


def _on(cache, stream):
    """The stream to launch on; the library launches on the current device, which must be the cache's."""
    if torch._C._cuda_getDevice() != cache._index:
        _refuse(cache, ())
    # (a stream is a few attribute look-ups away in torch.cuda; a step of small calls feels them)
    return torch._C._cuda_getCurrentRawStream(cache._index) if stream is None else _stream(stream)


def _check_rows(cache, k, v, row_offsets, starts):
    dtype = k.dtype
    if dtype not in _DTYPES:
        raise ValueError(f"unsupported dtype {dtype}")
    rows, b = (k.shape[0], *cache._row), cache.batch
    if not (_fits(cache, k, dtype, rows) and _fits(cache, v, dtype, rows)
            and _fits(cache, row_offsets, torch.int32, (b + 1,)) and _fits(cache, starts, torch.int32, (b,))):
        _refuse(cache, (("k", k, dtype, rows), ("v", v, dtype, rows),
                        ("row_offsets", row_offsets, torch.int32, (b + 1,)), ("starts", starts, torch.int32, (b,))))


def cache_write(cache, k, v, row_offsets, starts, stream=None):
    """Quantises the jagged rows of k and v [rows, kv_heads, head_dim] (bf16 or
    float32) into the cache: row t of sequence b goes to slot starts[b] + t
    (ba_cache_write)."""
    _check_rows(cache, k, v, row_offsets, starts)
    st = _load().ba_cache_write(cache._ref, _DTYPES[k.dtype], k.data_ptr(), v.data_ptr(), row_offsets.data_ptr(),
                                starts.data_ptr(), k.shape[0], _on(cache, stream))
    if st != BA_OK:
        raise BAError(st, "ba_cache_write")


def cache_read(cache, row_offsets, starts, total_rows, dtype=torch.bfloat16, k=None, v=None, stream=None):
    """Slots back as dense, jagged rows (k, v) [total_rows, kv_heads, head_dim]:
    row t of sequence b is slot starts[b] + t (ba_cache_read). Allocates k and
    v with torch unless both are given."""
    if (k is None) != (v is None):
        raise ValueError("pass both k and v, or neither")
    if k is None:
        k, v = (_empty((total_rows, *cache._row), dtype, cache.device, stream) for _ in "kv")
    _check_rows(cache, k, v, row_offsets, starts)
    if k.shape[0] != total_rows:
        raise ValueError(f"k and v must have {total_rows} rows")
    st = _load().ba_cache_read(cache._ref, _DTYPES[k.dtype], row_offsets.data_ptr(), starts.data_ptr(), total_rows,
                               k.data_ptr(), v.data_ptr(), _on(cache, stream))
    if st != BA_OK:
        raise BAError(st, "ba_cache_read")
    return k, v


def cache_summarize(cache, starts, ends, summaries, stream=None):
    """Mean keys of the full pages that hold a slot in [starts[b], ends[b]) into
    summaries, float32 [num_pages, kv_heads, head_dim] (ba_cache_summarize)."""
    b, shape = (cache.batch,), (cache.struct.num_pages, *cache._row)
    if not (_fits(cache, starts, torch.int32, b) and _fits(cache, ends, torch.int32, b)
            and _fits(cache, summaries, torch.float32, shape)):
        _refuse(cache, (("starts", starts, torch.int32, b), ("ends", ends, torch.int32, b),
                        ("summaries", summaries, torch.float32, shape)))
    st = _load().ba_cache_summarize(cache._ref, starts.data_ptr(), ends.data_ptr(), summaries.data_ptr(),
                                    _on(cache, stream))
    if st != BA_OK:
        raise BAError(st, "ba_cache_summarize")
    return summaries


def _check_queries(cache, q, q_offsets, lens, positions):
    """The queries' problem, after their checks."""
    if q.dim() != 3 or q.shape[1] % cache._row[0]:
        raise ValueError("q must be [rows, heads, head_dim] with heads a multiple of the cache's kv_heads")
    rows, heads, _ = q.shape
    b, shape = cache.batch, (rows, heads, cache._row[1])
    if not (_fits(cache, q, torch.bfloat16, shape) and _fits(cache, q_offsets, torch.int32, (b + 1,))
            and _fits(cache, lens, torch.int32, (b,))
            and (positions is None or _fits(cache, positions, torch.int32, (rows,)))):
        named = [("q", q, torch.bfloat16, shape), ("q_offsets", q_offsets, torch.int32, (b + 1,)),
                 ("lens", lens, torch.int32, (b,))]
        _refuse(cache, named if positions is None else [*named, ("positions", positions, torch.int32, (rows,))])
    return BAProblem(b, rows, heads, shape[2], BA_BF16)


def cache_select(cache, q, q_offsets, lens, summaries, block, window, topk, positions=None, page_mask=None,
                 stream=None):
    """The topk pages outside each query's window whose mean keys score highest,
    as bits, int32 [rows, kv_heads, ceil(max_pages / 32)] (ba_cache_select);
    allocates page_mask with torch."""
    prob = _check_queries(cache, q, q_offsets, lens, positions)
    kv_heads = cache._row[0]
    words, means = (prob.total_tokens, kv_heads, cache._words), (cache.struct.num_pages, *cache._row)
    if page_mask is None:
        page_mask = _empty(words, torch.int32, cache.device, stream)
    if not (_fits(cache, summaries, torch.float32, means) and _fits(cache, page_mask, torch.int32, words)):
        _refuse(cache, (("summaries", summaries, torch.float32, means), ("page_mask", page_mask, torch.int32, words)))
    st = _load().ba_cache_select(cache._ref, ctypes.byref(prob), q.data_ptr(), q_offsets.data_ptr(), lens.data_ptr(),
                                 _ptr(positions), summaries.data_ptr(), block, window, topk, page_mask.data_ptr(),
                                 _on(cache, stream))
    if st != BA_OK:
        raise BAError(st, "ba_cache_select")
    return page_mask


def cache_attention_fwd(cache, q, q_offsets, lens, block, window, positions=None, tree_mask=None, page_mask=None,
                        out=None, lse=None, workspace=None, stream=None):
    """Attention of new events over the cache under the block rule (ba_cache_fwd):
    one event a sequence, a chunk, a tree (tree_mask int32 [rows, words], and
    positions) or candidates, with pages selected outside the window
    (page_mask, from cache_select). Their own keys and values must be in the
    slots from lens on. Allocates out/lse (and a workspace) with torch."""
    prob = _check_queries(cache, q, q_offsets, lens, positions)
    rows, heads = prob.total_tokens, prob.heads
    if out is None:
        out = _empty(q.shape, torch.bfloat16, cache.device, stream)
    if lse is None:
        lse = _empty((heads, rows), torch.float32, cache.device, stream)
    named = [("out", out, torch.bfloat16, q.shape), ("lse", lse, torch.float32, (heads, rows))]
    words = 0
    if tree_mask is not None:
        if tree_mask.dim() != 2:
            raise ValueError("tree_mask must be [rows, words]")
        words = tree_mask.shape[1]
        if words < 1:
            raise ValueError("tree_mask must have a word a row")
        named.append(("tree_mask", tree_mask, torch.int32, (rows, words)))
    if page_mask is not None:
        named.append(("page_mask", page_mask, torch.int32, (rows, cache._row[0], cache._words)))
    for _, t, dtype, shape in named:
        if not _fits(cache, t, dtype, shape):
            _refuse(cache, named)
    ref = ctypes.byref(prob)
    if workspace is None:
        need = _load().ba_cache_fwd_workspace_size(cache._ref, ref, block, window)
        workspace = workspace_for(need, cache.device, stream)
    elif workspace.get_device() != cache._index or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on {cache.device}")
    st = _load().ba_cache_fwd(cache._ref, ref, q.data_ptr(), q_offsets.data_ptr(), lens.data_ptr(), _ptr(positions),
                              _ptr(tree_mask), words, _ptr(page_mask), block, window, out.data_ptr(), lse.data_ptr(),
                              workspace.data_ptr(), workspace.numel() * workspace.element_size(), _on(cache, stream))
    if st != BA_OK:
        raise BAError(st, "ba_cache_fwd")
    return out, lse
