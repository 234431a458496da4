"""Python binding of ``libfa.so``, the fused tiled attention library for B200 (sm_100a).

The functions carry the C names of ``include/fa.h`` and only marshal arguments: they check
dtypes, shapes and devices of torch tensors, allocate outputs when none are given (torch is the
device-memory allocator here), and pass raw pointers and sizes to the C ABI.  Every step of the
computation runs in the library's CUDA kernels.  If ``libfa.so`` is missing or cannot be loaded,
every call raises; there is no fallback.
"""
from __future__ import annotations

import contextlib
import ctypes
import importlib.util
import math
import os

__all__ = ["FaError", "lib", "fa_fwd", "fa_bwd", "fa_bwd_workspace_bytes", "fa_decode_int8", "fa_decode_int8_paged",
           "fa_decode_int4", "fa_decode_int4_paged", "fa_decode_int8_workspace_bytes",
           "fa_kv_quantize_int8", "fa_kv_quantize_int4", "fa_kv_dequantize_int8", "fa_kv_dequantize_int4",
           "fa_kv_append_int8_paged", "fa_kv_append_int4_paged", "fa_kv_gather_int8_paged",
           "fa_kv_gather_int4_paged", "fa_decode_int8_shared", "fa_decode_int4_shared",
           "fa_decode_shared_workspace_bytes",
           "fa_status_string", "fa_device_status", "fa_selftest_bounded_wait", "LIB_PATH",
           "STATUS"]

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libfa.so")

STATUS = {
    "FA_OK": 0,
    "FA_ERR_INVALID_ARG": -1,
    "FA_ERR_UNSUPPORTED": -2,
    "FA_ERR_ALIGNMENT": -3,
    "FA_ERR_WORKSPACE": -4,
    "FA_ERR_CUDA": -5,
    "FA_ERR_TIMEOUT": -6,
    "FA_ERR_DEVICE_INDEX": -7,
}


class FaError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {fa_status_string(status)} ({status})")


_lib = None
_P = ctypes.c_void_p
_I = ctypes.c_int
_F = ctypes.c_float
_Z = ctypes.c_size_t


def lib() -> ctypes.CDLL:
    """The loaded C library, with argument types declared.  Raises if it is not built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"libfa.so is not built ({LIB_PATH}); run "
                               "`python tiled_attention_26_b200/build.py`")
        L = ctypes.CDLL(LIB_PATH)
        L.fa_fwd.argtypes = [_P, _P, _P, _P, _P] + [_I] * 6 + [_F, _I, _I, _P]
        L.fa_fwd.restype = _I
        L.fa_fwd_ext.argtypes = ([_P, _P, _P, _P, _P] + [_I] * 6 + [_F, _I, _I, _I, _P,
                                 ctypes.c_int64, ctypes.c_int64, _P])
        L.fa_fwd_ext.restype = _I
        L.fa_bwd_workspace_bytes.argtypes = [_I, _I, _I]
        L.fa_bwd_workspace_bytes.restype = _Z
        L.fa_bwd.argtypes = [_P] * 9 + [_I] * 6 + [_F, _I, _I, _P, _Z, _P]
        L.fa_bwd.restype = _I
        L.fa_decode_int8_workspace_bytes.argtypes = [_I, _I, _I, _I]
        L.fa_decode_int8_workspace_bytes.restype = _Z
        L.fa_decode_int8.argtypes = [_P] * 7 + [_I] * 5 + [_F, _I, _P, _Z, _P]
        L.fa_decode_int8.restype = _I
        L.fa_decode_int8_paged.argtypes = [_P] * 9 + [_I] * 7 + [_F, _I, _P, _Z, _P]
        L.fa_decode_int8_paged.restype = _I
        L.fa_decode_int4.argtypes = [_P] * 7 + [_I] * 5 + [_F, _I, _P, _Z, _P]
        L.fa_decode_int4.restype = _I
        L.fa_decode_int4_paged.argtypes = [_P] * 9 + [_I] * 7 + [_F, _I, _P, _Z, _P]
        L.fa_decode_int4_paged.restype = _I
        for bits in (8, 4):
            f = getattr(L, f"fa_kv_quantize_int{bits}")
            f.argtypes, f.restype = [_P] * 6 + [_I] * 4 + [_P], _I
            f = getattr(L, f"fa_kv_dequantize_int{bits}")
            f.argtypes, f.restype = [_P] * 6 + [_I] * 4 + [_P], _I
            f = getattr(L, f"fa_kv_append_int{bits}_paged")
            f.argtypes = [_P, _P, ctypes.c_int64, ctypes.c_int64] + [_P] * 7 + [_I] * 7 + [_P]
            f.restype = _I
            f = getattr(L, f"fa_kv_gather_int{bits}_paged")
            f.argtypes, f.restype = [_P] * 9 + [_I] * 7 + [_P], _I
            f = getattr(L, f"fa_decode_int{bits}_shared")
            f.argtypes, f.restype = [_P] * 11 + [_I] * 8 + [_F, _I, _P, _Z, _P], _I
        L.fa_decode_shared_workspace_bytes.argtypes = [_I] * 7
        L.fa_decode_shared_workspace_bytes.restype = _Z
        L.fa_status_string.argtypes = [_I]
        L.fa_status_string.restype = ctypes.c_char_p
        L.fa_device_status.argtypes = [_P]
        L.fa_device_status.restype = _I
        L.fa_selftest_bounded_wait.argtypes = [_I, _P]
        L.fa_selftest_bounded_wait.restype = _I
        _lib = L
    return _lib


_CALLS = ["fa_kv_quantize_int8", "fa_kv_quantize_int4", "fa_kv_dequantize_int8",
          "fa_kv_dequantize_int4", "fa_kv_append_int8_paged", "fa_kv_append_int4_paged",
          "fa_kv_gather_int8_paged", "fa_kv_gather_int4_paged", "fa_decode_int8_shared",
          "fa_decode_int4_shared", "fa_decode_shared_workspace_bytes"]
_direct_calls = None


def _direct():
    """The direct calls of csrc/torch_calls.cpp: each makes the plain case of its entry point's call,
    or returns None and leaves it to the code here."""
    global _direct_calls
    if _direct_calls is None:
        L = lib()
        import torch  # noqa: F401  (its libraries must be loaded first)
        from .build import calls_path
        path = calls_path()
        if not os.path.exists(path):
            raise RuntimeError(f"the direct calls are not built for this torch and Python ({path}); run "
                               "`python tiled_attention_26_b200/build.py`")
        spec = importlib.util.spec_from_file_location(__name__ + "._torch_calls", path)
        calls = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(calls)
        calls.init(*(ctypes.cast(getattr(L, n), ctypes.c_void_p).value for n in _CALLS))
        _direct_calls = calls
    return _direct_calls


def fa_status_string(status: int) -> str:
    return lib().fa_status_string(int(status)).decode()


def _stream_ptr(stream):
    import torch
    if stream is None:
        return _current_stream_ptr(torch.cuda.current_device())
    return stream.cuda_stream


def _current_stream_ptr(index):
    """The current stream of device ``index``, as its pointer alone (a Stream object costs
    microseconds)."""
    import torch
    return torch._C._cuda_getCurrentRawStream(index)


def _check(t, name, dtype, shape, device):
    try:  # (tens of checks a step: the usual case without building a message or a tuple)
        if t.dtype is dtype and t.shape == shape and t.device == device and t.is_contiguous():
            return
    except AttributeError:
        pass
    import torch
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.device != device:
        raise ValueError(f"{name} must be on {device}, got {t.device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def fa_fwd(q, k, v, causal: bool = False, window: int = 0, scale: float | None = None,
           o=None, lse=None, return_lse: bool = True, stream=None, n_global: int = 0,
           mask=None):
    """Attention forward.  q: bf16 [B, Sq, Hq, D] on CUDA; k, v: bf16 [B, Skv, Hkv, D].
    ``n_global``: the first n_global positions attend to, and are attended by, every position.
    ``mask``: optional fp32 additive mask [Bm, Hm, Sq, Skv] with Bm in {1, B}, Hm in {1, Hq}
    (size-1 dims broadcast), added to scale * q.k; -inf drops a key.

    Returns ``(o, lse)``: o bf16 [B, Sq, Hq, D], lse fp32 [B, Hq, Sq] (natural log; None when
    ``return_lse`` is false and no ``lse`` buffer is given)."""
    import torch
    if q.dim() != 4 or k.dim() != 4:
        raise ValueError("q, k, v must be 4-D [B, S, H, D]")
    B, Sq, Hq, D = q.shape
    Skv, Hkv = k.shape[1], k.shape[2]
    dev = q.device
    _check(q, "q", torch.bfloat16, (B, Sq, Hq, D), dev)
    _check(k, "k", torch.bfloat16, (B, Skv, Hkv, D), dev)
    _check(v, "v", torch.bfloat16, (B, Skv, Hkv, D), dev)
    if o is None:
        o = torch.empty_like(q)
    _check(o, "o", torch.bfloat16, (B, Sq, Hq, D), dev)
    if lse is None and return_lse:
        lse = torch.empty((B, Hq, Sq), dtype=torch.float32, device=dev)
    if lse is not None:
        _check(lse, "lse", torch.float32, (B, Hq, Sq), dev)
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    sb = sh = 0
    if mask is not None:
        if mask.dim() != 4 or mask.shape[0] not in (1, B) or mask.shape[1] not in (1, Hq):
            raise ValueError("mask must be [1 or B, 1 or Hq, Sq, Skv]")
        _check(mask, "mask", torch.float32, (mask.shape[0], mask.shape[1], Sq, Skv), dev)
        sh = Sq * Skv if mask.shape[1] == Hq else 0
        sb = Sq * Skv * mask.shape[1] if mask.shape[0] == B else 0
    rc = lib().fa_fwd_ext(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(),
                          lse.data_ptr() if lse is not None else None, B, Hq, Hkv, Sq, Skv, D,
                          float(scale), int(bool(causal)), int(window), int(n_global),
                          mask.data_ptr() if mask is not None else None, sb, sh,
                          _stream_ptr(stream))
    if rc != 0:
        raise FaError(rc, "fa_fwd")
    return o, lse


def fa_bwd_workspace_bytes(B: int, Hq: int, Sq: int) -> int:
    return int(lib().fa_bwd_workspace_bytes(int(B), int(Hq), int(Sq)))


def fa_bwd(q, k, v, o, dout, lse, causal: bool = False, window: int = 0,
           scale: float | None = None, dq=None, dk=None, dv=None, workspace=None, stream=None):
    """Backward pass of fa_fwd: gradients of sum(dout * o).  q, o, dout: bf16 [B, Sq, Hq, D];
    k, v: bf16 [B, Skv, Hkv, D]; lse: fp32 [B, Hq, Sq] from fa_fwd.  Returns (dq, dk, dv)."""
    import torch
    B, Sq, Hq, D = q.shape
    Skv, Hkv = k.shape[1], k.shape[2]
    dev = q.device
    _check(q, "q", torch.bfloat16, (B, Sq, Hq, D), dev)
    _check(k, "k", torch.bfloat16, (B, Skv, Hkv, D), dev)
    _check(v, "v", torch.bfloat16, (B, Skv, Hkv, D), dev)
    _check(o, "o", torch.bfloat16, (B, Sq, Hq, D), dev)
    _check(dout, "dout", torch.bfloat16, (B, Sq, Hq, D), dev)
    _check(lse, "lse", torch.float32, (B, Hq, Sq), dev)
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    _check(dq, "dq", torch.bfloat16, (B, Sq, Hq, D), dev)
    _check(dk, "dk", torch.bfloat16, (B, Skv, Hkv, D), dev)
    _check(dv, "dv", torch.bfloat16, (B, Skv, Hkv, D), dev)
    need = fa_bwd_workspace_bytes(B, Hq, Sq)
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=dev)
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    rc = lib().fa_bwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), dout.data_ptr(),
                      lse.data_ptr(), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), B, Hq, Hkv,
                      Sq, Skv, D, float(scale), int(bool(causal)), int(window),
                      workspace.data_ptr(), workspace.numel() * workspace.element_size(),
                      _stream_ptr(stream))
    if rc != 0:
        raise FaError(rc, "fa_bwd")
    return dq, dk, dv


def fa_decode_int8_workspace_bytes(B: int, Hq: int, D: int, num_splits: int) -> int:
    return int(lib().fa_decode_int8_workspace_bytes(int(B), int(Hq), int(D), int(num_splits)))


def _decode(bits, q, k, v, k_scale, v_scale, num_splits, scale, o, lse, workspace, return_lse,
            stream):
    import torch
    name = f"fa_decode_int{bits}"
    B, one, Hq, D = q.shape
    if one != 1:
        raise ValueError("decode takes one query token per sequence")
    Skv, Hkv = k.shape[1], k.shape[2]
    dev = q.device
    code = torch.int8 if bits == 8 else torch.uint8
    row = D if bits == 8 else D // 2
    _check(q, "q", torch.bfloat16, (B, 1, Hq, D), dev)
    _check(k, "k", code, (B, Skv, Hkv, row), dev)
    _check(v, "v", code, (B, Skv, Hkv, row), dev)
    _check(k_scale, "k_scale", torch.float32, (B, Hkv, Skv), dev)
    _check(v_scale, "v_scale", torch.float32, (B, Hkv, Skv), dev)
    if o is None:
        o = torch.empty_like(q)
    _check(o, "o", torch.bfloat16, (B, 1, Hq, D), dev)
    if lse is None and return_lse:
        lse = torch.empty((B, Hq), dtype=torch.float32, device=dev)
    if lse is not None:
        _check(lse, "lse", torch.float32, (B, Hq), dev)
    need = fa_decode_int8_workspace_bytes(B, Hq, D, num_splits)
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=dev)
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    rc = getattr(lib(), name)(q.data_ptr(), k.data_ptr(), v.data_ptr(), k_scale.data_ptr(),
                              v_scale.data_ptr(), o.data_ptr(),
                              lse.data_ptr() if lse is not None else None, B, Hq, Hkv, Skv, D,
                              float(scale), int(num_splits), workspace.data_ptr(),
                              workspace.numel() * workspace.element_size(), _stream_ptr(stream))
    if rc != 0:
        raise FaError(rc, name)
    return o, lse


def fa_decode_int8(q, k, v, k_scale, v_scale, num_splits: int = 16, scale: float | None = None,
                   o=None, lse=None, workspace=None, return_lse: bool = True, stream=None):
    """Decode step over an INT8 KV cache.  q: bf16 [B, 1, Hq, D]; k, v: int8 [B, Skv, Hkv, D];
    k_scale, v_scale: fp32 [B, Hkv, Skv].  Returns ``(o, lse)`` with o bf16 [B, 1, Hq, D] and
    lse fp32 [B, Hq]."""
    return _decode(8, q, k, v, k_scale, v_scale, num_splits, scale, o, lse, workspace,
                   return_lse, stream)


def fa_decode_int4(q, k, v, k_scale, v_scale, num_splits: int = 16, scale: float | None = None,
                   o=None, lse=None, workspace=None, return_lse: bool = True, stream=None):
    """Decode step over an INT4 KV cache.  k, v: uint8 [B, Skv, Hkv, D/2], two 4-bit
    two's-complement codes per byte (dim 2i in the low nibble); otherwise as fa_decode_int8."""
    return _decode(4, q, k, v, k_scale, v_scale, num_splits, scale, o, lse, workspace,
                   return_lse, stream)


def _decode_paged(bits, q, k_pages, v_pages, k_scale_pages, v_scale_pages, block_table, seqlens,
                  num_splits, scale, o, lse, workspace, return_lse, stream):
    import torch
    name = f"fa_decode_int{bits}_paged"
    B, one, Hq, D = q.shape
    if one != 1:
        raise ValueError("decode takes one query token per sequence")
    if k_pages.dim() != 4 or block_table.dim() != 2:
        raise ValueError("k_pages must be [num_pages, P, Hkv, row], block_table [B, max_pages]")
    num_pages, P, Hkv = k_pages.shape[0], k_pages.shape[1], k_pages.shape[2]
    max_pages = block_table.shape[1]
    dev = q.device
    code = torch.int8 if bits == 8 else torch.uint8
    row = D if bits == 8 else D // 2
    _check(q, "q", torch.bfloat16, (B, 1, Hq, D), dev)
    _check(k_pages, "k_pages", code, (num_pages, P, Hkv, row), dev)
    _check(v_pages, "v_pages", code, (num_pages, P, Hkv, row), dev)
    _check(k_scale_pages, "k_scale_pages", torch.float32, (num_pages, Hkv, P), dev)
    _check(v_scale_pages, "v_scale_pages", torch.float32, (num_pages, Hkv, P), dev)
    _check(block_table, "block_table", torch.int32, (B, max_pages), dev)
    _check(seqlens, "seqlens", torch.int32, (B,), dev)
    if o is None:
        o = torch.empty_like(q)
    _check(o, "o", torch.bfloat16, (B, 1, Hq, D), dev)
    if lse is None and return_lse:
        lse = torch.empty((B, Hq), dtype=torch.float32, device=dev)
    if lse is not None:
        _check(lse, "lse", torch.float32, (B, Hq), dev)
    need = fa_decode_int8_workspace_bytes(B, Hq, D, num_splits)
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=dev)
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    rc = getattr(lib(), name)(
        q.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(), k_scale_pages.data_ptr(),
        v_scale_pages.data_ptr(), block_table.data_ptr(), seqlens.data_ptr(), o.data_ptr(),
        lse.data_ptr() if lse is not None else None, B, Hq, Hkv, P, max_pages, num_pages, D,
        float(scale), int(num_splits), workspace.data_ptr(),
        workspace.numel() * workspace.element_size(), _stream_ptr(stream))
    if rc != 0:
        raise FaError(rc, name)
    return o, lse


def fa_decode_int8_paged(q, k_pages, v_pages, k_scale_pages, v_scale_pages, block_table,
                         seqlens, num_splits: int = 16, scale: float | None = None, o=None,
                         lse=None, workspace=None, return_lse: bool = True, stream=None):
    """Decode step over a paged INT8 KV cache with one length per sequence.
    q: bf16 [B, 1, Hq, D]; k_pages, v_pages: int8 [num_pages, P, Hkv, D]; k_scale_pages,
    v_scale_pages: fp32 [num_pages, Hkv, P]; block_table: int32 [B, max_pages]; seqlens: int32
    [B] (both on the device).  Returns ``(o, lse)`` with o bf16 [B, 1, Hq, D], lse fp32 [B, Hq]."""
    return _decode_paged(8, q, k_pages, v_pages, k_scale_pages, v_scale_pages, block_table,
                         seqlens, num_splits, scale, o, lse, workspace, return_lse, stream)


def fa_decode_int4_paged(q, k_pages, v_pages, k_scale_pages, v_scale_pages, block_table,
                         seqlens, num_splits: int = 16, scale: float | None = None, o=None,
                         lse=None, workspace=None, return_lse: bool = True, stream=None):
    """Paged, variable-length decode over an INT4 KV cache: k_pages, v_pages uint8
    [num_pages, P, Hkv, D/2] packed as for fa_decode_int4; otherwise as fa_decode_int8_paged."""
    return _decode_paged(4, q, k_pages, v_pages, k_scale_pages, v_scale_pages, block_table,
                         seqlens, num_splits, scale, o, lse, workspace, return_lse, stream)


_HERE = contextlib.nullcontext()


def _on(dev, stream):
    """Context in which a call's buffers are allocated and its kernels launched: the tensors'
    device, and ``stream`` (whose device it must be) where one is given, so that a buffer the call
    allocates belongs to the stream that uses it."""
    import torch
    if dev.type != "cuda":
        raise ValueError(f"tensors must be on a CUDA device, got {dev}")
    if stream is not None:
        if stream.device != dev:
            raise ValueError(f"stream is on {stream.device}, the tensors are on {dev}")
        return torch.cuda.stream(stream)
    return _HERE if torch.cuda.current_device() == dev.index else torch.cuda.device(dev)


def _buffer(t, name, dtype, shape, like):
    """The caller's output ``t``, checked, or a new one on the device of ``like``."""
    if t is None:
        return like.new_empty(shape, dtype=dtype)
    _check(t, name, dtype, shape, like.device)
    return t


def _code_type(bits, D):
    """dtype and elements of one row of D codes."""
    import torch
    return (torch.int8, D) if bits == 8 else (torch.uint8, D // 2)


def _kv_quantize(bits, k, v, k_codes, v_codes, k_scale, v_scale, stream):
    if stream is None:
        r = _direct().kv_quantize(bits, k, v, k_codes, v_codes, k_scale, v_scale)
        if r is not None:
            if r[0] != 0:
                raise FaError(r[0], f"fa_kv_quantize_int{bits}")
            return r[1:]
    import torch
    name = f"fa_kv_quantize_int{bits}"
    if k.dim() != 4:
        raise ValueError("k, v must be 4-D [B, S, Hkv, D]")
    B, S, Hkv, D = k.shape
    dev = k.device
    code, row = _code_type(bits, D)
    _check(k, "k", torch.bfloat16, (B, S, Hkv, D), dev)
    _check(v, "v", torch.bfloat16, (B, S, Hkv, D), dev)
    with _on(dev, stream):
        out = (_buffer(k_codes, "k_codes", code, (B, S, Hkv, row), k),
               _buffer(v_codes, "v_codes", code, (B, S, Hkv, row), k),
               _buffer(k_scale, "k_scale", torch.float32, (B, Hkv, S), k),
               _buffer(v_scale, "v_scale", torch.float32, (B, Hkv, S), k))
        rc = getattr(lib(), name)(k.data_ptr(), v.data_ptr(), *(t.data_ptr() for t in out), B, S,
                                  Hkv, D, _current_stream_ptr(dev.index))
    if rc != 0:
        raise FaError(rc, name)
    return out


def fa_kv_quantize_int8(k, v, k_codes=None, v_codes=None, k_scale=None, v_scale=None, stream=None):
    """Quantise whole K and V caches for fa_decode_int8.  k, v: bf16 [B, S, Hkv, D].  Returns
    ``(k_codes, v_codes, k_scale, v_scale)``: int8 [B, S, Hkv, D] twice, fp32 [B, Hkv, S] twice
    (the buffers given, or new ones)."""
    return _kv_quantize(8, k, v, k_codes, v_codes, k_scale, v_scale, stream)


def fa_kv_quantize_int4(k, v, k_codes=None, v_codes=None, k_scale=None, v_scale=None, stream=None):
    """As fa_kv_quantize_int8 for fa_decode_int4: codes uint8 [B, S, Hkv, D/2], two per byte."""
    return _kv_quantize(4, k, v, k_codes, v_codes, k_scale, v_scale, stream)


def _kv_dequantize(bits, k_codes, v_codes, k_scale, v_scale, k, v, stream):
    if stream is None:
        r = _direct().kv_dequantize(bits, k_codes, v_codes, k_scale, v_scale, k, v)
        if r is not None:
            if r[0] != 0:
                raise FaError(r[0], f"fa_kv_dequantize_int{bits}")
            return r[1:]
    import torch
    name = f"fa_kv_dequantize_int{bits}"
    if k_codes.dim() != 4:
        raise ValueError("k_codes, v_codes must be 4-D [B, S, Hkv, row]")
    B, S, Hkv, row = k_codes.shape
    D = row if bits == 8 else 2 * row
    dev = k_codes.device
    code, _ = _code_type(bits, D)
    _check(k_codes, "k_codes", code, (B, S, Hkv, row), dev)
    _check(v_codes, "v_codes", code, (B, S, Hkv, row), dev)
    _check(k_scale, "k_scale", torch.float32, (B, Hkv, S), dev)
    _check(v_scale, "v_scale", torch.float32, (B, Hkv, S), dev)
    with _on(dev, stream):
        k = _buffer(k, "k", torch.bfloat16, (B, S, Hkv, D), k_codes)
        v = _buffer(v, "v", torch.bfloat16, (B, S, Hkv, D), k_codes)
        rc = getattr(lib(), name)(k_codes.data_ptr(), v_codes.data_ptr(), k_scale.data_ptr(),
                                  v_scale.data_ptr(), k.data_ptr(), v.data_ptr(), B, S, Hkv, D,
                                  _current_stream_ptr(dev.index))
    if rc != 0:
        raise FaError(rc, name)
    return k, v


def fa_kv_dequantize_int8(k_codes, v_codes, k_scale, v_scale, k=None, v=None, stream=None):
    """Read a cache of fa_kv_quantize_int8 back: ``(k, v)`` bf16 [B, S, Hkv, D] = code * scale."""
    return _kv_dequantize(8, k_codes, v_codes, k_scale, v_scale, k, v, stream)


def fa_kv_dequantize_int4(k_codes, v_codes, k_scale, v_scale, k=None, v=None, stream=None):
    """Read a cache of fa_kv_quantize_int4 back: ``(k, v)`` bf16 [B, S, Hkv, D] = code * scale."""
    return _kv_dequantize(4, k_codes, v_codes, k_scale, v_scale, k, v, stream)


def _check_pool(bits, D, k_pages, v_pages, k_scale_pages, v_scale_pages, block_table, dev, B=None):
    """Checks a page pool and a block table; returns (num_pages, P, Hkv, B, max_pages)."""
    import torch
    if k_pages.dim() != 4 or block_table.dim() != 2:
        raise ValueError("k_pages must be [num_pages, P, Hkv, row], block_table [B, max_pages]")
    num_pages, P, Hkv, _ = k_pages.shape
    B, max_pages = (block_table.shape[0] if B is None else B), block_table.shape[1]
    code, row = _code_type(bits, D)
    _check(k_pages, "k_pages", code, (num_pages, P, Hkv, row), dev)
    _check(v_pages, "v_pages", code, (num_pages, P, Hkv, row), dev)
    _check(k_scale_pages, "k_scale_pages", torch.float32, (num_pages, Hkv, P), dev)
    _check(v_scale_pages, "v_scale_pages", torch.float32, (num_pages, Hkv, P), dev)
    _check(block_table, "block_table", torch.int32, (B, max_pages), dev)
    return num_pages, P, Hkv, B, max_pages


def _token_rows(t, name, Hkv, D, dev):
    """Number of token rows of t ([N, Hkv, D] or [B, T, Hkv, D], each row contiguous, rows evenly
    spaced) and the elements between them."""
    import torch
    if not isinstance(t, torch.Tensor) or t.dtype != torch.bfloat16:
        raise TypeError(f"{name} must be a torch.bfloat16 tensor")
    if t.dim() not in (3, 4) or tuple(t.shape[-2:]) != (Hkv, D):
        raise ValueError(f"{name} must have shape [N, {Hkv}, {D}] or [B, T, {Hkv}, {D}], got {tuple(t.shape)}")
    if t.device != dev:
        raise ValueError(f"{name} must be on {dev}, got {t.device}")
    if t.numel() == 0:
        return 0, Hkv * D
    st = t.stride()
    if (st[-1] != 1 and D > 1) or (st[-2] != D and Hkv > 1):
        raise ValueError(f"{name}: each token's [Hkv, D] row must be contiguous")
    n, step = t.shape[0], st[0]
    if t.dim() == 4:
        n, step = t.shape[0] * t.shape[1], st[1]
        if t.shape[1] == 1:
            step = st[0]
        elif t.shape[0] > 1 and st[0] != t.shape[1] * st[1]:
            raise ValueError(f"{name}: token rows must be evenly spaced")
    return n, (step if n > 1 else max(step, Hkv * D))


def _kv_append(bits, k, v, k_pages, v_pages, k_scale_pages, v_scale_pages, block_table, positions,
               cu_tokens, stream):
    if stream is None:
        rc = _direct().kv_append(bits, k, v, k_pages, v_pages, k_scale_pages, v_scale_pages,
                                 block_table, positions, cu_tokens)
        if rc is not None:
            if rc != 0:
                raise FaError(rc, f"fa_kv_append_int{bits}_paged")
            return
    import torch
    name = f"fa_kv_append_int{bits}_paged"
    dev, D = k.device, k.shape[-1]
    num_pages, P, Hkv, B, max_pages = _check_pool(bits, D, k_pages, v_pages, k_scale_pages,
                                                  v_scale_pages, block_table, dev)
    n, k_stride = _token_rows(k, "k", Hkv, D, dev)
    nv, v_stride = _token_rows(v, "v", Hkv, D, dev)
    if v.shape != k.shape:
        raise ValueError(f"v must have shape {tuple(k.shape)}, got {tuple(v.shape)}")
    if positions is not None:
        _check(positions, "positions", torch.int32, (B,), dev)
    if cu_tokens is not None:
        _check(cu_tokens, "cu_tokens", torch.int32, (B + 1,), dev)
    elif k.dim() == 4 and k.shape[0] != B:
        raise ValueError(f"k must hold {B} sequences, got {k.shape[0]}")
    with _on(dev, stream):
        rc = getattr(lib(), name)(
            k.data_ptr(), v.data_ptr(), k_stride, v_stride, k_pages.data_ptr(), v_pages.data_ptr(),
            k_scale_pages.data_ptr(), v_scale_pages.data_ptr(), block_table.data_ptr(),
            positions.data_ptr() if positions is not None else None,
            cu_tokens.data_ptr() if cu_tokens is not None else None, n, B, Hkv, P, max_pages,
            num_pages, D, _current_stream_ptr(dev.index))
    if rc != 0:
        raise FaError(rc, name)


def fa_kv_append_int8_paged(k, v, k_pages, v_pages, k_scale_pages, v_scale_pages, block_table,
                            positions=None, cu_tokens=None, stream=None):
    """Quantise new tokens into a paged INT8 cache (the layout of fa_decode_int8_paged), in place.
    k, v: bf16 [N, Hkv, D] or [B, T, Hkv, D]; token rows may be strided (slices of one projection's
    output).  positions: int32 [B], each sequence's length before the call (None: 0).  cu_tokens:
    int32 [B + 1], first row of each sequence's new tokens (None: the same number of each)."""
    _kv_append(8, k, v, k_pages, v_pages, k_scale_pages, v_scale_pages, block_table, positions,
               cu_tokens, stream)


def fa_kv_append_int4_paged(k, v, k_pages, v_pages, k_scale_pages, v_scale_pages, block_table,
                            positions=None, cu_tokens=None, stream=None):
    """As fa_kv_append_int8_paged into uint8 [num_pages, P, Hkv, D/2] pages of fa_decode_int4_paged."""
    _kv_append(4, k, v, k_pages, v_pages, k_scale_pages, v_scale_pages, block_table, positions,
               cu_tokens, stream)


def _kv_gather(bits, k_pages, v_pages, k_scale_pages, v_scale_pages, block_table, num_tokens,
               positions, cu_tokens, k, v, stream):
    if stream is None:
        r = _direct().kv_gather(bits, k_pages, v_pages, k_scale_pages, v_scale_pages, block_table,
                                num_tokens, positions, cu_tokens, k, v)
        if r is not None:
            if r[0] != 0:
                raise FaError(r[0], f"fa_kv_gather_int{bits}_paged")
            return r[1:]
    import torch
    name = f"fa_kv_gather_int{bits}_paged"
    dev = k_pages.device
    D = k_pages.shape[-1] * (1 if bits == 8 else 2)
    num_pages, P, Hkv, B, max_pages = _check_pool(bits, D, k_pages, v_pages, k_scale_pages,
                                                  v_scale_pages, block_table, dev)
    if positions is not None:
        _check(positions, "positions", torch.int32, (B,), dev)
    if cu_tokens is not None:
        _check(cu_tokens, "cu_tokens", torch.int32, (B + 1,), dev)
    n = int(num_tokens)
    if n < 0:
        raise ValueError(f"num_tokens must not be negative, got {n}")
    with _on(dev, stream):
        k = _buffer(k, "k", torch.bfloat16, (n, Hkv, D), k_pages)
        v = _buffer(v, "v", torch.bfloat16, (n, Hkv, D), k_pages)
        rc = getattr(lib(), name)(
            k_pages.data_ptr(), v_pages.data_ptr(), k_scale_pages.data_ptr(),
            v_scale_pages.data_ptr(), block_table.data_ptr(),
            positions.data_ptr() if positions is not None else None,
            cu_tokens.data_ptr() if cu_tokens is not None else None, k.data_ptr(), v.data_ptr(),
            n, B, Hkv, P, max_pages, num_pages, D, _current_stream_ptr(dev.index))
    if rc != 0:
        raise FaError(rc, name)
    return k, v


def fa_kv_gather_int8_paged(k_pages, v_pages, k_scale_pages, v_scale_pages, block_table, num_tokens,
                            positions=None, cu_tokens=None, k=None, v=None, stream=None):
    """Read ``num_tokens`` tokens of a paged INT8 cache back as ``(k, v)``, bf16 [num_tokens, Hkv, D]
    each: row cu_tokens[b] + i is position positions[b] + i of sequence b (positions None: 0;
    cu_tokens None: num_tokens / B of each sequence).  Rows behind cu_tokens[B] are left as they
    were (undefined in new buffers)."""
    return _kv_gather(8, k_pages, v_pages, k_scale_pages, v_scale_pages, block_table, num_tokens,
                      positions, cu_tokens, k, v, stream)


def fa_kv_gather_int4_paged(k_pages, v_pages, k_scale_pages, v_scale_pages, block_table, num_tokens,
                            positions=None, cu_tokens=None, k=None, v=None, stream=None):
    """As fa_kv_gather_int8_paged from a paged INT4 cache."""
    return _kv_gather(4, k_pages, v_pages, k_scale_pages, v_scale_pages, block_table, num_tokens,
                      positions, cu_tokens, k, v, stream)


def fa_decode_shared_workspace_bytes(B: int, Hq: int, Hkv: int, D: int, max_prefix_len: int,
                                     max_seqlen: int, num_splits: int = 0) -> int:
    return int(lib().fa_decode_shared_workspace_bytes(B, Hq, Hkv, D, max_prefix_len, max_seqlen,
                                                      num_splits))


def _decode_shared(bits, q, k_pages, v_pages, k_scale_pages, v_scale_pages, prefix_table,
                   prefix_len, block_table, seqlens, num_splits, scale, o, lse, workspace,
                   return_lse, stream):
    if stream is None:
        r = _direct().decode_shared(bits, q, k_pages, v_pages, k_scale_pages, v_scale_pages,
                                    prefix_table, prefix_len, block_table, seqlens, num_splits, scale,
                                    o, lse, workspace, return_lse)
        if r is not None:
            if r[0] != 0:
                raise FaError(r[0], f"fa_decode_int{bits}_shared")
            return r[1:]
    import torch
    name = f"fa_decode_int{bits}_shared"
    if q.dim() != 4 or q.shape[1] != 1:
        raise ValueError("decode takes one query token per sequence, q [B, 1, Hq, D]")
    B, _, Hq, D = q.shape
    dev = q.device
    _check(q, "q", torch.bfloat16, (B, 1, Hq, D), dev)
    num_pages, P, Hkv, _, max_pages = _check_pool(bits, D, k_pages, v_pages, k_scale_pages,
                                                  v_scale_pages, block_table, dev, B)
    if prefix_table.dim() != 1:
        raise ValueError("prefix_table must be [max_prefix_pages]")
    max_prefix = prefix_table.shape[0]
    _check(prefix_table, "prefix_table", torch.int32, (max_prefix,), dev)
    _check(prefix_len, "prefix_len", torch.int32, (1,), dev)
    _check(seqlens, "seqlens", torch.int32, (B,), dev)
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    with _on(dev, stream):
        o = _buffer(o, "o", torch.bfloat16, (B, 1, Hq, D), q)
        if lse is not None or return_lse:
            lse = _buffer(lse, "lse", torch.float32, (B, Hq), q)
        if workspace is None:
            need = lib().fa_decode_shared_workspace_bytes(B, Hq, Hkv, D, max_prefix * P,
                                                          max_pages * P, num_splits)
            workspace = q.new_empty(max(need, 1), dtype=torch.uint8)
        elif workspace.device != dev or not workspace.is_contiguous():
            raise ValueError(f"workspace must be contiguous and on {dev}")
        rc = getattr(lib(), name)(
            q.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(), k_scale_pages.data_ptr(),
            v_scale_pages.data_ptr(), prefix_table.data_ptr(), prefix_len.data_ptr(),
            block_table.data_ptr(), seqlens.data_ptr(), o.data_ptr(),
            lse.data_ptr() if lse is not None else None, B, Hq, Hkv, P, max_prefix, max_pages,
            num_pages, D, scale, num_splits, workspace.data_ptr(),
            workspace.numel() * workspace.element_size(), _current_stream_ptr(dev.index))
    if rc != 0:
        raise FaError(rc, name)
    return o, lse


def fa_decode_int8_shared(q, k_pages, v_pages, k_scale_pages, v_scale_pages, prefix_table,
                          prefix_len, block_table, seqlens, num_splits: int = 0,
                          scale: float | None = None, o=None, lse=None, workspace=None,
                          return_lse: bool = True, stream=None):
    """Decode step of a batch that shares a prefix, over a paged INT8 cache.  prefix_table: int32
    [max_prefix_pages] and prefix_len: int32 [1], the shared keys' pages and number; block_table:
    int32 [B, max_pages] and seqlens: int32 [B], each sequence's own keys (all on the device).
    num_splits: splits of the own keys (0: chosen).  Otherwise as fa_decode_int8_paged; returns
    ``(o, lse)``."""
    return _decode_shared(8, q, k_pages, v_pages, k_scale_pages, v_scale_pages, prefix_table,
                          prefix_len, block_table, seqlens, num_splits, scale, o, lse, workspace,
                          return_lse, stream)


def fa_decode_int4_shared(q, k_pages, v_pages, k_scale_pages, v_scale_pages, prefix_table,
                          prefix_len, block_table, seqlens, num_splits: int = 0,
                          scale: float | None = None, o=None, lse=None, workspace=None,
                          return_lse: bool = True, stream=None):
    """As fa_decode_int8_shared over uint8 [num_pages, P, Hkv, D/2] pages of fa_decode_int4_paged."""
    return _decode_shared(4, q, k_pages, v_pages, k_scale_pages, v_scale_pages, prefix_table,
                          prefix_len, block_table, seqlens, num_splits, scale, o, lse, workspace,
                          return_lse, stream)


def fa_device_status(stream=None) -> int:
    return int(lib().fa_device_status(_stream_ptr(stream)))


def fa_selftest_bounded_wait(timeout_us: int, stream=None) -> int:
    return int(lib().fa_selftest_bounded_wait(int(timeout_us), _stream_ptr(stream)))
