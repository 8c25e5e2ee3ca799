"""Python binding of the MiMo-V2-Flash hybrid attention library (sm_100a).

Argument marshalling only: every step of the computation runs in the CUDA
kernels of ``libmimo_attn.so`` (C ABI in ``include/mimo_attn.h``).  PyTorch is
used for device memory and the current stream.  There is no fallback: if the
library cannot be loaded, importing this package raises.

Entry points (same names as the C ABI):

* ``mimo_attn_prefill(q, k, v, sinks, window, cu_seqlens, max_seqlen, ...)``
* ``mimo_attn_decode(q, k_cache, v_cache, seqlens, window, sinks, ...)``
* ``mimo_attn_paged_attention(q, k_pages, v_pages, block_table, cu_seqlens_q, seqlens, ...)``
  with ``mimo_attn_paged_append``, ``mimo_attn_page_hold``, ``mimo_attn_page_fork``,
  ``mimo_attn_page_compact`` and ``mimo_attn_page_copy``: the paged cache
  (``paged_cache.PagedCache`` keeps one)
* ``mimo_attn_decode_workspace_size(...)``, ``mimo_attn_device_status(...)``
"""

from __future__ import annotations

import contextlib
import ctypes
import functools
import importlib.machinery
import math
import os

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
#: MIMO_ATTN_CHECKED=1 in the environment loads the bounds-checked build
#: (libmimo_attn_checked.so: every kernel checks its row indices, see the header)
CHECKED = os.environ.get("MIMO_ATTN_CHECKED", "0") not in ("", "0")
LIB_PATH = os.path.join(_PKG, "libmimo_attn_checked.so" if CHECKED else "libmimo_attn.so")

MIMO_OK = 0
MIMO_ERR_INVALID_ARG = 1
MIMO_ERR_UNSUPPORTED = 2
MIMO_ERR_CUDA = 3
MIMO_ERR_WORKSPACE = 4
MIMO_ERR_TIMEOUT = 5
MIMO_ERR_BOUNDS = 6
MIMO_DTYPE_BF16 = 0
MIMO_DTYPE_F32 = 1

#: entry points declared in include/mimo_attn.h
EXPORTED = (
    "mimo_attn_prefill",
    "mimo_attn_decode_workspace_size",
    "mimo_attn_decode",
    "mimo_attn_last_error",
    "mimo_attn_device_status",
    "mimo_attn_set_device_status",
    "mimo_attn_decode_noalloc",
    "mimo_attn_decode_fp8_workspace_size",
    "mimo_attn_decode_fp8",
    "mimo_attn_rope_append",
    "mimo_attn_decode_merge",
    "mimo_attn_prefill_backward_workspace_size",
    "mimo_attn_prefill_backward",
    "mimo_attn_paged_attention_workspace_size",
    "mimo_attn_paged_attention",
    "mimo_attn_paged_append",
    "mimo_attn_page_hold_workspace_size",
    "mimo_attn_page_hold",
    "mimo_attn_page_fork",
    "mimo_attn_page_compact_workspace_size",
    "mimo_attn_page_compact",
    "mimo_attn_page_copy",
    "mimo_attn_wait_selftest",
    "mimo_attn_is_checked_build",
    "mimo_attn_checked_site",
    "mimo_attn_checked_selftest",
)


class MimoAttnError(RuntimeError):
    def __init__(self, status, msg):
        super().__init__(f"mimo_attn status {status}: {msg}")
        self.status = status


class Dims(ctypes.Structure):
    _fields_ = [
        ("num_heads_q", ctypes.c_int),
        ("num_heads_kv", ctypes.c_int),
        ("head_dim_qk", ctypes.c_int),
        ("head_dim_v", ctypes.c_int),
        ("softmax_scale", ctypes.c_float),
        ("v_scale", ctypes.c_float),
        ("out_dtype", ctypes.c_int),
    ]


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            f"{LIB_PATH} is missing; build it with global_attention_swa_b200._build.build("
            f"{'checked=True' if CHECKED else ''})")
    lib = ctypes.CDLL(LIB_PATH)
    vp, i32, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
    dp = ctypes.POINTER(Dims)
    lib.mimo_attn_prefill.argtypes = [dp, vp, vp, vp, vp, i32, vp, i32, i32, i32, vp, vp, vp]
    lib.mimo_attn_prefill.restype = i32
    lib.mimo_attn_decode_workspace_size.argtypes = [dp, i32, i32, i32]
    lib.mimo_attn_decode_workspace_size.restype = sz
    lib.mimo_attn_decode.argtypes = [dp, vp, vp, vp, vp, i32, i32, i32, vp, vp, vp, vp, sz, vp]
    lib.mimo_attn_decode.restype = i32
    lib.mimo_attn_last_error.argtypes = []
    lib.mimo_attn_last_error.restype = ctypes.c_char_p
    lib.mimo_attn_device_status.argtypes = [vp]
    lib.mimo_attn_device_status.restype = i32
    lib.mimo_attn_set_device_status.argtypes = [i32, vp]
    lib.mimo_attn_set_device_status.restype = i32
    lib.mimo_attn_decode_fp8_workspace_size.argtypes = [dp, i32, i32, i32]
    lib.mimo_attn_decode_fp8_workspace_size.restype = sz
    lib.mimo_attn_decode_fp8.argtypes = [dp, vp, vp, vp, vp, vp, vp, i32, i32, i32, vp, vp, vp, vp,
                                         sz, vp]
    lib.mimo_attn_decode_fp8.restype = i32
    lib.mimo_attn_rope_append.argtypes = [dp, vp, vp, vp, vp, vp, vp, i32, i32, i32,
                                          ctypes.c_float, i32, vp]
    lib.mimo_attn_rope_append.restype = i32
    lib.mimo_attn_decode_merge.argtypes = [dp, vp, vp, i32, i32, vp, vp, vp, vp]
    lib.mimo_attn_decode_merge.restype = i32
    lib.mimo_attn_prefill_backward_workspace_size.argtypes = [dp, i32]
    lib.mimo_attn_prefill_backward_workspace_size.restype = sz
    lib.mimo_attn_prefill_backward.argtypes = [dp, vp, vp, vp, vp, vp, vp, vp, i32, vp, i32, i32, i32,
                                               vp, vp, vp, vp, vp, sz, vp]
    lib.mimo_attn_prefill_backward.restype = i32
    lib.mimo_attn_paged_attention_workspace_size.argtypes = [dp, i32, i32, i32, i32]
    lib.mimo_attn_paged_attention_workspace_size.restype = sz
    lib.mimo_attn_paged_attention.argtypes = [dp, vp, vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, i32,
                                              i32, vp, vp, vp, vp, sz, vp]
    lib.mimo_attn_paged_attention.restype = i32
    lib.mimo_attn_paged_append.argtypes = [dp, vp, vp, vp, vp, vp, vp, vp, vp, vp, i32, i32, i32, i32, i32,
                                           ctypes.c_float, i32, vp]
    lib.mimo_attn_paged_append.restype = i32
    lib.mimo_attn_page_hold_workspace_size.argtypes = [i32]
    lib.mimo_attn_page_hold_workspace_size.restype = sz
    lib.mimo_attn_page_hold.argtypes = [vp, i32, vp, i32, i32, i32, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    lib.mimo_attn_page_hold.restype = i32
    lib.mimo_attn_page_fork.argtypes = [vp, i32, vp, i32, i32, vp, i32, vp, vp, vp]
    lib.mimo_attn_page_fork.restype = i32
    lib.mimo_attn_page_compact_workspace_size.argtypes = [i32]
    lib.mimo_attn_page_compact_workspace_size.restype = sz
    lib.mimo_attn_page_compact.argtypes = [vp, i32, vp, i32, i32, i32, vp, vp, vp, vp, vp, sz, vp]
    lib.mimo_attn_page_compact.restype = i32
    lib.mimo_attn_page_copy.argtypes = [dp, vp, vp, i32, i32, i32, vp, i32, vp]
    lib.mimo_attn_page_copy.restype = i32
    lib.mimo_attn_wait_selftest.argtypes = [vp]
    lib.mimo_attn_wait_selftest.restype = i32
    lib.mimo_attn_is_checked_build.argtypes = []
    lib.mimo_attn_is_checked_build.restype = i32
    lib.mimo_attn_checked_site.argtypes = [vp]
    lib.mimo_attn_checked_site.restype = i32
    lib.mimo_attn_checked_selftest.argtypes = [vp]
    lib.mimo_attn_checked_selftest.restype = i32
    return lib


lib = _load()

if hasattr(lib, "mimo_attn_decode_noalloc"):
    lib.mimo_attn_decode_noalloc.argtypes = [ctypes.POINTER(Dims)] + [ctypes.c_void_p] * 4 + [
        ctypes.c_int, ctypes.c_int, ctypes.c_int] + [ctypes.c_void_p] * 4
    lib.mimo_attn_decode_noalloc.restype = ctypes.c_int


def _check(status):
    if status != MIMO_OK:
        raise MimoAttnError(status, lib.mimo_attn_last_error().decode())


_BF16, _F32, _I32 = torch.bfloat16, torch.float32, torch.int32
_OUT = (torch.bfloat16, torch.float32)


def _ptr(t, name="tensor", dtype=None):
    """Device address of a contiguous CUDA tensor (None for None).  The C ABI takes
    plain pointers, so a host tensor, a strided view or another dtype would be
    read as garbage: each is refused here."""
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype not in (dtype if isinstance(dtype, tuple) else (dtype,)):
        raise TypeError(f"{name} must be {dtype} (got {t.dtype})")
    return ctypes.c_void_p(t.data_ptr())


def _shape(t, shape, name):
    """Refuse a tensor whose shape disagrees with the sizes the call derives from
    its other arguments (the library would read or write past its end)."""
    if t is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")


def _same_device(dev, **tensors):
    """Refuse tensors that live on another device than the call's (the library
    launches on the current device and would dereference another GPU's memory)."""
    for name, t in tensors.items():
        if t is not None and t.device != dev:
            raise ValueError(f"{name} is on {t.device}, but the call runs on {dev}")


@contextlib.contextmanager
def _on_device(dev):
    """Make the tensors' device current for the call (launches, device queries)."""
    if dev.type == "cuda":
        with torch.cuda.device(dev):
            yield
    else:  # host tensors never reach the library: _ptr refuses them
        yield


def _stream(stream, dev):
    """The stream to launch on: the caller's (which must belong to dev) or dev's
    current stream."""
    if stream is None:
        if dev.index is not None:  # the handle alone, without a Stream object
            return ctypes.c_void_p(torch._C._cuda_getCurrentRawStream(dev.index))
        stream = torch.cuda.current_stream(dev)
    elif stream.device != dev:
        raise ValueError(f"stream belongs to {stream.device}, but the call runs on {dev}")
    return ctypes.c_void_p(stream.cuda_stream)


def make_dims(hq, hkv, dqk=192, dv=128, softmax_scale=None, v_scale=1.0, out_dtype=torch.bfloat16):
    return Dims(hq, hkv, dqk, dv,
                0.0 if softmax_scale is None else float(softmax_scale),
                float(v_scale),
                MIMO_DTYPE_F32 if out_dtype == torch.float32 else MIMO_DTYPE_BF16)


def mimo_attn_prefill(q, k, v, sinks, window, cu_seqlens, max_seqlen, out=None, lse=None,
                      out_dtype=torch.bfloat16, softmax_scale=None, v_scale=1.0,
                      return_lse=True, stream=None):
    """Packed varlen prefill.  q [Nt,Hq,192], k [Nt,Hkv,192], v [Nt,Hkv,128] bf16 (CUDA).

    Returns (out [Nt,Hq,128], lse [Hq,Nt] fp32 or None).
    """
    nt, hq, dqk = q.shape
    hkv, dv = k.shape[1], v.shape[2]
    _shape(k, (nt, hkv, dqk), "k")
    _shape(v, (nt, hkv, dv), "v")
    _shape(sinks, (hq,), "sinks")
    if cu_seqlens.dim() != 1 or cu_seqlens.numel() < 1:
        raise ValueError("cu_seqlens must be 1-D with num_seqs + 1 entries")
    _shape(out, (nt, hq, dv), "out")
    _shape(lse, (hq, nt), "lse")
    if out is None:
        out = torch.empty((nt, hq, dv), dtype=out_dtype, device=q.device)
    if lse is None and return_lse:
        lse = torch.empty((hq, nt), dtype=torch.float32, device=q.device)
    dev = q.device
    _same_device(dev, k=k, v=v, sinks=sinks, cu_seqlens=cu_seqlens, out=out, lse=lse)
    dims = make_dims(hq, hkv, dqk, dv, softmax_scale, v_scale, out.dtype)
    with _on_device(dev):
        _check(lib.mimo_attn_prefill(ctypes.byref(dims), _ptr(q, "q", _BF16), _ptr(k, "k", _BF16),
                                     _ptr(v, "v", _BF16), _ptr(sinks, "sinks", _F32), int(window),
                                     _ptr(cu_seqlens, "cu_seqlens", _I32), int(cu_seqlens.numel() - 1),
                                     nt, int(max_seqlen), _ptr(out, "out", _OUT),
                                     _ptr(lse, "lse", _F32), _stream(stream, dev)))
    return out, lse


def _decode_shapes(q, k_cache, v_cache, seqlens, sinks, out, lse):
    B, hq, dqk = q.shape
    if k_cache.dim() != 4 or v_cache.dim() != 4:
        raise ValueError("caches must be [batch, capacity, Hkv, D]")
    C, hkv = k_cache.shape[1], k_cache.shape[2]
    _shape(k_cache, (B, C, hkv, dqk), "k_cache")
    _shape(v_cache, (B, C, hkv, v_cache.shape[3]), "v_cache")
    _shape(seqlens, (B,), "seqlens")
    _shape(sinks, (hq,), "sinks")
    _shape(out, (B, hq, v_cache.shape[3]), "out")
    _shape(lse, (B, hq), "lse")


def mimo_attn_decode_workspace_size(hq, hkv, batch, capacity, window, dqk=192, dv=128):
    dims = make_dims(hq, hkv, dqk, dv)
    return int(lib.mimo_attn_decode_workspace_size(ctypes.byref(dims), batch, capacity, window))


def mimo_attn_decode(q, k_cache, v_cache, seqlens, window, sinks, out=None, lse=None,
                     workspace=None, out_dtype=torch.bfloat16, softmax_scale=None, v_scale=1.0,
                     return_lse=True, stream=None):
    """One decode step.  q [B,Hq,192]; caches [B,C,Hkv,192/128] bf16; seqlens [B] int32.

    Returns (out [B,Hq,128], lse [B,Hq] fp32 or None).
    """
    B, hq, dqk = q.shape
    C, hkv = k_cache.shape[1], k_cache.shape[2]
    dv = v_cache.shape[3]
    _decode_shapes(q, k_cache, v_cache, seqlens, sinks, out, lse)
    if out is None:
        out = torch.empty((B, hq, dv), dtype=out_dtype, device=q.device)
    if lse is None and return_lse:
        lse = torch.empty((B, hq), dtype=torch.float32, device=q.device)
    dev = q.device
    dims = make_dims(hq, hkv, dqk, dv, softmax_scale, v_scale, out.dtype)
    need = int(lib.mimo_attn_decode_workspace_size(ctypes.byref(dims), B, C, int(window)))
    if need and workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    _same_device(dev, k_cache=k_cache, v_cache=v_cache, seqlens=seqlens, sinks=sinks, out=out,
                 lse=lse, workspace=workspace)
    wbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    with _on_device(dev):
        _check(lib.mimo_attn_decode(ctypes.byref(dims), _ptr(q, "q", _BF16),
                                    _ptr(k_cache, "k_cache", _BF16), _ptr(v_cache, "v_cache", _BF16),
                                    _ptr(seqlens, "seqlens", _I32), B, C, int(window),
                                    _ptr(sinks, "sinks", _F32), _ptr(out, "out", _OUT),
                                    _ptr(lse, "lse", _F32), _ptr(workspace, "workspace"), wbytes,
                                    _stream(stream, dev)))
    return out, lse


def mimo_attn_decode_fp8(q, k_cache, v_cache, k_scale, v_scale_kv, seqlens, window, sinks,
                         out=None, lse=None, workspace=None, out_dtype=torch.bfloat16,
                         softmax_scale=None, v_scale=1.0, return_lse=True, stream=None):
    """One decode step against e4m3 caches.  q [B,Hq,192] bf16; caches [B,C,Hkv,192/128]
    as torch.float8_e4m3fn or uint8 codes; k_scale / v_scale_kv [Hkv] fp32.

    Returns (out [B,Hq,128], lse [B,Hq] fp32 or None).
    """
    B, hq, dqk = q.shape
    C, hkv = k_cache.shape[1], k_cache.shape[2]
    dv = v_cache.shape[3]
    if k_cache.element_size() != 1 or v_cache.element_size() != 1:
        raise TypeError("FP8 caches hold one byte per element")
    _decode_shapes(q, k_cache, v_cache, seqlens, sinks, out, lse)
    _shape(k_scale, (hkv,), "k_scale")
    _shape(v_scale_kv, (hkv,), "v_scale_kv")
    if out is None:
        out = torch.empty((B, hq, dv), dtype=out_dtype, device=q.device)
    if lse is None and return_lse:
        lse = torch.empty((B, hq), dtype=torch.float32, device=q.device)
    dev = q.device
    dims = make_dims(hq, hkv, dqk, dv, softmax_scale, v_scale, out.dtype)
    need = int(lib.mimo_attn_decode_fp8_workspace_size(ctypes.byref(dims), B, C, int(window)))
    if need and workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    _same_device(dev, k_cache=k_cache, v_cache=v_cache, k_scale=k_scale, v_scale_kv=v_scale_kv,
                 seqlens=seqlens, sinks=sinks, out=out, lse=lse, workspace=workspace)
    wbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    with _on_device(dev):
        _check(lib.mimo_attn_decode_fp8(ctypes.byref(dims), _ptr(q, "q", _BF16),
                                        _ptr(k_cache, "k_cache"), _ptr(v_cache, "v_cache"),
                                        _ptr(k_scale, "k_scale", _F32),
                                        _ptr(v_scale_kv, "v_scale_kv", _F32),
                                        _ptr(seqlens, "seqlens", _I32), B, C, int(window),
                                        _ptr(sinks, "sinks", _F32), _ptr(out, "out", _OUT),
                                        _ptr(lse, "lse", _F32), _ptr(workspace, "workspace"), wbytes,
                                        _stream(stream, dev)))
    return out, lse


def mimo_attn_rope_append(q, k_new, v_new, k_cache, v_cache, seqlens, window, rope_theta,
                          rotary_dim=None, stream=None):
    """Rotate the new token's q (in place) and k, and write k, v into the cache slot of
    position seqlens - 1 (see include/mimo_attn.h).  Returns q."""
    B, hq, dqk = q.shape
    C, hkv = k_cache.shape[1], k_cache.shape[2]
    _decode_shapes(q, k_cache, v_cache, seqlens, None, None, None)
    _shape(k_new, (B, hkv, dqk), "k_new")
    _shape(v_new, (B, hkv, v_cache.shape[3]), "v_new")
    dev = q.device
    _same_device(dev, k_new=k_new, v_new=v_new, k_cache=k_cache, v_cache=v_cache, seqlens=seqlens)
    dims = make_dims(hq, hkv, dqk, v_cache.shape[3])
    rd = dqk if rotary_dim is None else int(rotary_dim)
    with _on_device(dev):
        _check(lib.mimo_attn_rope_append(ctypes.byref(dims), _ptr(q, "q", _BF16),
                                         _ptr(k_new, "k_new", _BF16), _ptr(v_new, "v_new", _BF16),
                                         _ptr(k_cache, "k_cache", _BF16),
                                         _ptr(v_cache, "v_cache", _BF16),
                                         _ptr(seqlens, "seqlens", _I32), B, C, int(window),
                                         float(rope_theta), rd, _stream(stream, dev)))
    return q


def mimo_attn_decode_merge(part_out, part_lse, sinks, out=None, lse=None,
                           out_dtype=torch.bfloat16, v_scale=1.0, return_lse=True, stream=None):
    """Merge per-part decode results (part_out [R,B,Hq,128] fp32, part_lse [R,B,Hq] fp32)
    with the sink.  Returns (out [B,Hq,128], lse [B,Hq] or None)."""
    R, B, hq, dv = part_out.shape
    _shape(part_lse, (R, B, hq), "part_lse")
    _shape(sinks, (hq,), "sinks")
    _shape(out, (B, hq, dv), "out")
    _shape(lse, (B, hq), "lse")
    if out is None:
        out = torch.empty((B, hq, dv), dtype=out_dtype, device=part_out.device)
    if lse is None and return_lse:
        lse = torch.empty((B, hq), dtype=torch.float32, device=part_out.device)
    dev = part_out.device
    _same_device(dev, part_lse=part_lse, sinks=sinks, out=out, lse=lse)
    dims = make_dims(hq, 1, 192, dv, None, v_scale, out.dtype)
    with _on_device(dev):
        _check(lib.mimo_attn_decode_merge(ctypes.byref(dims), _ptr(part_out, "part_out", _F32),
                                          _ptr(part_lse, "part_lse", _F32), R, B,
                                          _ptr(sinks, "sinks", _F32), _ptr(out, "out", _OUT),
                                          _ptr(lse, "lse", _F32), _stream(stream, dev)))
    return out, lse


def mimo_attn_prefill_backward(q, k, v, out, lse, dout, sinks, window, cu_seqlens, max_seqlen,
                               softmax_scale=None, v_scale=1.0, stream=None):
    """Gradients of mimo_attn_prefill: returns (dq, dk, dv [fp32], dsinks [Hq] fp32 or None).

    ``out`` and ``lse`` are the forward's results; ``dout`` has out's dtype.
    """
    nt, hq, dqk = q.shape
    hkv, dv_dim = k.shape[1], v.shape[2]
    _shape(k, (nt, hkv, dqk), "k")
    _shape(v, (nt, hkv, dv_dim), "v")
    _shape(out, (nt, hq, dv_dim), "out")
    _shape(lse, (hq, nt), "lse")
    _shape(dout, (nt, hq, dv_dim), "dout")
    _shape(sinks, (hq,), "sinks")
    if cu_seqlens.dim() != 1 or cu_seqlens.numel() < 1:
        raise ValueError("cu_seqlens must be 1-D with num_seqs + 1 entries")
    dq = torch.empty((nt, hq, dqk), dtype=torch.float32, device=q.device)
    dk = torch.empty((nt, hkv, dqk), dtype=torch.float32, device=q.device)
    dv = torch.empty((nt, hkv, dv_dim), dtype=torch.float32, device=q.device)
    ds = None if sinks is None else torch.empty(hq, dtype=torch.float32, device=q.device)
    dev = q.device
    _same_device(dev, k=k, v=v, out=out, lse=lse, dout=dout, sinks=sinks, cu_seqlens=cu_seqlens)
    dims = make_dims(hq, hkv, dqk, dv_dim, softmax_scale, v_scale, out.dtype)
    need = int(lib.mimo_attn_prefill_backward_workspace_size(ctypes.byref(dims), nt))
    ws = torch.empty(max(need, 16), dtype=torch.uint8, device=dev)
    with _on_device(dev):
        _check(lib.mimo_attn_prefill_backward(ctypes.byref(dims), _ptr(q, "q", _BF16),
                                              _ptr(k, "k", _BF16), _ptr(v, "v", _BF16),
                                              _ptr(out, "out", _OUT), _ptr(lse, "lse", _F32),
                                              _ptr(dout, "dout", out.dtype),
                                              _ptr(sinks, "sinks", _F32), int(window),
                                              _ptr(cu_seqlens, "cu_seqlens", _I32),
                                              cu_seqlens.numel() - 1, nt, int(max_seqlen), _ptr(dq),
                                              _ptr(dk), _ptr(dv), _ptr(ds), _ptr(ws), ws.numel(),
                                              _stream(stream, dev)))
    return dq, dk, dv, ds


def _load_fast():
    """The native part of the binding (csrc/fast_call.cpp) on the loaded library, or None
    where it was not built: the calls then go through the marshalling below.  One that is
    there and does not load (built against another torch) is an error."""
    if not any(os.path.exists(os.path.join(_PKG, "_fast_call" + s)) for s in importlib.machinery.EXTENSION_SUFFIXES):
        return None
    from . import _fast_call

    _fast_call.bind(*(ctypes.cast(getattr(lib, f"mimo_attn_{name}"), ctypes.c_void_p).value for name in (
        "paged_attention", "paged_attention_workspace_size", "paged_append", "page_hold",
        "page_hold_workspace_size", "page_fork", "page_compact", "page_compact_workspace_size", "page_copy")))
    return _fast_call


_fast = _load_fast()


def _taken(r):
    """The result of a native call: its tensors, or the error its status stands for."""
    if r.__class__ is int:
        _check(r)
    return r


_dims_ref = functools.lru_cache(maxsize=256)(lambda *args: ctypes.byref(make_dims(*args)))


def _addr(t, name, dtype, shape, dev):
    """Device address (0 for None) of a contiguous CUDA tensor of this dtype and shape on
    dev: _shape, _same_device and _ptr in one look for the common case, and by their own
    words where something is wrong."""
    if t is None:
        return 0
    if t.shape == shape and t.dtype is dtype and t.device == dev and t.is_contiguous() and t.is_cuda:
        return t.data_ptr()
    _shape(t, shape, name)
    _same_device(dev, **{name: t})
    return _ptr(t, name, dtype).value


def _call(fn, dev, *args):
    """fn(*args, stream) with the tensors' device current; args[-1] is the caller's stream."""
    *args, stream = args
    stream = _stream(stream, dev)
    if dev.type != "cuda" or torch.cuda.current_device() == dev.index:
        status = fn(*args, stream)
    else:
        with torch.cuda.device(dev):
            status = fn(*args, stream)
    if status:
        _check(status)


def _int(x, name):
    """x as the C int that the library takes (ctypes would cut it to 32 bits)."""
    x = int(x)
    if not -2 ** 31 <= x < 2 ** 31:
        raise ValueError(f"{name} is out of range (got {x})")
    return x


def _new(like, shape, stream, dtype=None):
    """An uninitialised tensor beside ``like`` for a call on ``stream`` (None: the current
    one).  Its memory comes from that stream's, so no work still pending elsewhere writes
    it; and it is not given out again before the current stream, where the caller reads
    the result, has come past its end."""
    if stream is None or not like.is_cuda:
        return like.new_empty(shape, dtype=dtype)
    current = torch.cuda.current_stream(like.device)
    with torch.cuda.stream(stream):
        t = like.new_empty(shape, dtype=dtype)
    t.record_stream(current)
    return t


def _other_stream(stream, *tensors):
    """Tensors that are used on ``stream``, wherever they were made: their memory is not
    given out again before ``stream`` is past the call."""
    if stream is not None:
        for t in tensors:
            if t is not None:
                t.record_stream(stream)


def _paged_pools(k_pages, v_pages, block_table):
    """(num_pages, page_size, Hkv, Dqk, Dv, num_seqs, max_pages) of a paged cache."""
    if k_pages.dim() != 4 or v_pages.dim() != 4:
        raise ValueError("k_pages and v_pages must be [num_pages, page_size, Hkv, D]")
    if block_table.dim() != 2:
        raise ValueError("block_table must be [num_seqs, max_pages]")
    return (*k_pages.shape, v_pages.shape[3], *block_table.shape)


def mimo_attn_paged_attention_workspace_size(hq, hkv, num_seqs, total_q, max_seqlen_q, window=0, dqk=192,
                                             dv=128):
    dims = make_dims(hq, hkv, dqk, dv)
    return int(lib.mimo_attn_paged_attention_workspace_size(ctypes.byref(dims), num_seqs, total_q,
                                                            max_seqlen_q, window))


def mimo_attn_paged_attention(q, k_pages, v_pages, block_table, cu_seqlens_q, seqlens, max_seqlen_q,
                              window, sinks, out=None, lse=None, workspace=None,
                              out_dtype=torch.bfloat16, softmax_scale=None, v_scale=1.0,
                              return_lse=True, stream=None):
    """Attention of each sequence's new tokens over its paged cache (chunked prefill,
    drafted tokens, decode; see include/mimo_attn.h).  q [Nt,Hq,192] bf16 packed by
    cu_seqlens_q [B+1]; k_pages / v_pages [P,page_size,Hkv,192/128] bf16; block_table
    [B,max_pages] and seqlens [B] (the new tokens included) int32.

    Returns (out [Nt,Hq,128], lse [Hq,Nt] fp32 or None).
    """
    if _fast is not None and stream is None and (out is not None or out_dtype in _OUT):
        r = _fast.paged_attention(q, k_pages, v_pages, block_table, cu_seqlens_q, seqlens, max_seqlen_q, window,
                                  sinks, out, lse, workspace, (out_dtype if out is None else out.dtype) is _F32,
                                  0.0 if softmax_scale is None else softmax_scale, v_scale, return_lse)
        if r is not None:
            return _taken(r)
    nt, hq, dqk = q.shape
    P, ps, hkv, _, dv, B, M = _paged_pools(k_pages, v_pages, block_table)
    dev = q.device
    addrs = (_addr(q, "q", _BF16, (nt, hq, dqk), dev), _addr(k_pages, "k_pages", _BF16, (P, ps, hkv, dqk), dev),
             _addr(v_pages, "v_pages", _BF16, (P, ps, hkv, dv), dev),
             _addr(block_table, "block_table", _I32, (B, M), dev),
             _addr(cu_seqlens_q, "cu_seqlens_q", _I32, (B + 1,), dev), _addr(seqlens, "seqlens", _I32, (B,), dev))
    sink = _addr(sinks, "sinks", _F32, (hq,), dev)
    if out is None:
        out = _new(q, (nt, hq, dv), stream, out_dtype)
    if lse is None and return_lse:
        lse = _new(q, (hq, nt), stream, _F32)
    max_seqlen_q, window = _int(max_seqlen_q, "max_seqlen_q"), _int(window, "window")
    dims = _dims_ref(hq, hkv, dqk, dv, None if softmax_scale is None else float(softmax_scale), float(v_scale),
                     out.dtype)
    need = lib.mimo_attn_paged_attention_workspace_size(dims, B, nt, max_seqlen_q, window)
    ws = wbytes = 0
    if workspace is not None:
        ws = _addr(workspace, "workspace", workspace.dtype, workspace.shape, dev)
        wbytes = workspace.numel() * workspace.element_size()
    elif need:
        workspace, wbytes = _new(block_table, need + 3 >> 2, stream), need
        ws = workspace.data_ptr()
    _call(lib.mimo_attn_paged_attention, dev, dims, *addrs, B, nt, max_seqlen_q, P, ps, M, window, sink,
          _addr(out, "out", out.dtype if out.dtype in _OUT else _OUT, (nt, hq, dv), dev),
          _addr(lse, "lse", _F32, (hq, nt), dev), ws, wbytes, stream)
    _other_stream(stream, out, lse, workspace)
    return out, lse


def mimo_attn_paged_append(q, k_new, v_new, k_pages, v_pages, block_table, cu_seqlens_q, seqlens,
                           rope_theta, rotary_dim=None, q_out=None, stream=None):
    """Rotate the new tokens' q and k and write k, v into their pages (see
    include/mimo_attn.h).  Returns the rotated q: ``q_out`` (which may be q), or a new tensor."""
    if _fast is not None and stream is None:
        r = _fast.paged_append(q, k_new, v_new, k_pages, v_pages, block_table, cu_seqlens_q, seqlens, rope_theta,
                               q.shape[-1] if rotary_dim is None else rotary_dim, q_out)
        if r is not None:
            return _taken(r)
    nt, hq, dqk = q.shape
    P, ps, hkv, _, dv, B, M = _paged_pools(k_pages, v_pages, block_table)
    dev = q.device
    if q_out is None:
        q_out = _new(q, (nt, hq, dqk), stream)
    _call(lib.mimo_attn_paged_append, dev, _dims_ref(hq, hkv, dqk, dv),
          _addr(q, "q", _BF16, (nt, hq, dqk), dev), _addr(q_out, "q_out", _BF16, (nt, hq, dqk), dev),
          _addr(k_new, "k_new", _BF16, (nt, hkv, dqk), dev), _addr(v_new, "v_new", _BF16, (nt, hkv, dv), dev),
          _addr(k_pages, "k_pages", _BF16, (P, ps, hkv, dqk), dev),
          _addr(v_pages, "v_pages", _BF16, (P, ps, hkv, dv), dev),
          _addr(block_table, "block_table", _I32, (B, M), dev),
          _addr(cu_seqlens_q, "cu_seqlens_q", _I32, (B + 1,), dev), _addr(seqlens, "seqlens", _I32, (B,), dev),
          B, nt, P, ps, M, float(rope_theta), dqk if rotary_dim is None else _int(rotary_dim, "rotary_dim"), stream)
    _other_stream(stream, q_out)
    return q_out


def _page_table(page_refs, block_table):
    if page_refs.dim() != 1 or block_table.dim() != 2:
        raise ValueError("page_refs must be [num_pages] and block_table [num_seqs, max_pages]")
    return (page_refs.shape[0], *block_table.shape)


def _page_workspace(workspace, need, like, stream):
    """(tensor, address, bytes) of the caller's workspace, or of a new one beside ``like``."""
    if workspace is None:
        workspace = _new(like, need + 3 >> 2, stream)
        return workspace, workspace.data_ptr(), need
    return (workspace, _addr(workspace, "workspace", workspace.dtype, workspace.shape, like.device),
            workspace.numel() * workspace.element_size())


def mimo_attn_page_hold(page_refs, block_table, seqlens, page_size, first=None, write_from=None,
                        refs_out=None, table_out=None, moves=None, info=None, workspace=None,
                        stream=None):
    """Make each sequence hold exactly the pages of positions [first, seqlens), those from
    write_from on its own (see include/mimo_attn.h).  refs_out / table_out may be
    page_refs / block_table (in place); None allocates them.

    Returns (refs_out, table_out, moves [B,2] for mimo_attn_page_copy, info [2]: pages
    missing (nothing was changed if > 0), pages free afterwards).
    """
    if _fast is not None and stream is None:
        r = _fast.page_hold(page_refs, block_table, seqlens, page_size, first, write_from, refs_out, table_out, moves,
                            info, workspace)
        if r is not None:
            return _taken(r)
    P, B, M = _page_table(page_refs, block_table)
    dev = page_refs.device
    refs_out = _new(page_refs, (P,), stream) if refs_out is None else refs_out
    table_out = _new(page_refs, (B, M), stream) if table_out is None else table_out
    moves = _new(page_refs, (B, 2), stream) if moves is None else moves
    info = _new(page_refs, (2,), stream) if info is None else info
    ws, ws_addr, ws_bytes = _page_workspace(workspace, lib.mimo_attn_page_hold_workspace_size(P), page_refs, stream)
    _call(lib.mimo_attn_page_hold, dev, _addr(page_refs, "page_refs", _I32, (P,), dev), P,
          _addr(block_table, "block_table", _I32, (B, M), dev), B, M, _int(page_size, "page_size"),
          _addr(seqlens, "seqlens", _I32, (B,), dev), _addr(first, "first", _I32, (B,), dev),
          _addr(write_from, "write_from", _I32, (B,), dev), _addr(refs_out, "refs_out", _I32, (P,), dev),
          _addr(table_out, "table_out", _I32, (B, M), dev), _addr(moves, "moves", _I32, (B, 2), dev),
          _addr(info, "info", _I32, (2,), dev), ws_addr, ws_bytes, stream)
    _other_stream(stream, refs_out, table_out, moves, info, ws)
    return refs_out, table_out, moves, info


def mimo_attn_page_fork(page_refs, block_table, parent, refs_out=None, table_out=None, stream=None):
    """Row i of the new table is row parent[i] of block_table, empty where parent[i] < 0
    (see include/mimo_attn.h).  refs_out may be page_refs (in place); table_out may not
    be block_table.  Returns (refs_out, table_out)."""
    if _fast is not None and stream is None:
        r = _fast.page_fork(page_refs, block_table, parent, refs_out, table_out)
        if r is not None:
            return _taken(r)
    if parent.dim() != 1:
        raise ValueError("parent must be 1-D")
    P, B, M = _page_table(page_refs, block_table)
    n = parent.shape[0]
    dev = page_refs.device
    refs_out = _new(page_refs, (P,), stream) if refs_out is None else refs_out
    table_out = _new(page_refs, (n, M), stream) if table_out is None else table_out
    _call(lib.mimo_attn_page_fork, dev, _addr(page_refs, "page_refs", _I32, (P,), dev), P,
          _addr(block_table, "block_table", _I32, (B, M), dev), B, M, _addr(parent, "parent", _I32, (n,), dev), n,
          _addr(refs_out, "refs_out", _I32, (P,), dev), _addr(table_out, "table_out", _I32, (n, M), dev), stream)
    _other_stream(stream, refs_out, table_out)
    return refs_out, table_out


def mimo_attn_page_compact(page_refs, block_table, max_moves, refs_out=None, table_out=None,
                           moves=None, info=None, workspace=None, stream=None):
    """Give the used pages at the end of the pool the free places at its front, at most
    max_moves of them (see include/mimo_attn.h).  refs_out / table_out may be the inputs.

    Returns (refs_out, table_out, moves [max_moves,2] for mimo_attn_page_copy, info [2]:
    moves made, pages in use).
    """
    if _fast is not None and stream is None:
        r = _fast.page_compact(page_refs, block_table, max_moves, refs_out, table_out, moves, info, workspace)
        if r is not None:
            return _taken(r)
    P, B, M = _page_table(page_refs, block_table)
    max_moves = _int(max_moves, "max_moves")
    dev = page_refs.device
    refs_out = _new(page_refs, (P,), stream) if refs_out is None else refs_out
    table_out = _new(page_refs, (B, M), stream) if table_out is None else table_out
    moves = _new(page_refs, (max_moves, 2), stream) if moves is None else moves
    info = _new(page_refs, (2,), stream) if info is None else info
    ws, ws_addr, ws_bytes = _page_workspace(workspace, lib.mimo_attn_page_compact_workspace_size(P), page_refs, stream)
    _call(lib.mimo_attn_page_compact, dev, _addr(page_refs, "page_refs", _I32, (P,), dev), P,
          _addr(block_table, "block_table", _I32, (B, M), dev), B, M, max_moves,
          _addr(refs_out, "refs_out", _I32, (P,), dev), _addr(table_out, "table_out", _I32, (B, M), dev),
          _addr(moves, "moves", _I32, (max_moves, 2), dev), _addr(info, "info", _I32, (2,), dev), ws_addr,
          ws_bytes, stream)
    _other_stream(stream, refs_out, table_out, moves, info, ws)
    return refs_out, table_out, moves, info


def mimo_attn_page_copy(k_pages, v_pages, moves, stream=None):
    """Copy pages moves[:, 0] over pages moves[:, 1] in place (rows of -1 are skipped; see
    include/mimo_attn.h).  k_pages / v_pages [P,page_size,Hkv,192/128] bf16 of one layer, or
    [layers,P,...] of several.  Returns (k_pages, v_pages)."""
    if _fast is not None and stream is None:
        r = _fast.page_copy(k_pages, v_pages, moves)
        if r is not None:
            return _taken(r)
    if k_pages.dim() not in (4, 5) or k_pages.dim() != v_pages.dim():
        raise ValueError("k_pages and v_pages must be [num_pages, page_size, Hkv, D], or with a layer axis first")
    shape = k_pages.shape
    P, ps, hkv, dqk = shape[-4:]
    dv, n, dev = v_pages.shape[-1], moves.shape[0], k_pages.device
    _call(lib.mimo_attn_page_copy, dev, _dims_ref(hkv, hkv, dqk, dv), _addr(k_pages, "k_pages", _BF16, shape, dev),
          _addr(v_pages, "v_pages", _BF16, (*shape[:-1], dv), dev), shape[0] if len(shape) == 5 else 1, P, ps,
          _addr(moves, "moves", _I32, (n, 2), dev), n, stream)
    return k_pages, v_pages


def _current_device():
    return torch.device("cuda", torch.cuda.current_device())


def mimo_attn_device_status(stream=None, device=None):
    """Synchronise the stream (default: the current stream of ``device``, itself
    defaulting to the current device); raise if a kernel recorded a device-side
    error on that device."""
    dev = torch.device(device) if device is not None else (
        stream.device if stream is not None else _current_device())
    with _on_device(dev):
        _check(lib.mimo_attn_device_status(_stream(stream, dev)))


def mimo_attn_set_device_status(code, stream=None, device=None):
    """Pre-load the device status word (test hook for the failure path; see
    include/mimo_attn.h)."""
    dev = torch.device(device) if device is not None else (
        stream.device if stream is not None else _current_device())
    with _on_device(dev):
        _check(lib.mimo_attn_set_device_status(int(code), _stream(stream, dev)))


def mimo_attn_wait_selftest(stream=None, device=None):
    """Failure-path test hook: a kernel whose wait runs out after its bound
    (about 1 s) and records MIMO_ERR_TIMEOUT (see include/mimo_attn.h)."""
    dev = torch.device(device) if device is not None else (
        stream.device if stream is not None else _current_device())
    with _on_device(dev):
        _check(lib.mimo_attn_wait_selftest(_stream(stream, dev)))


def mimo_attn_is_checked_build():
    """True when the loaded library is the bounds-checked build."""
    return bool(lib.mimo_attn_is_checked_build())


def mimo_attn_checked_site(stream=None, device=None):
    """Synchronise the stream; return (and clear) the first site at which the
    checked build caught a row index outside its buffer, 0 if none; raise if a
    CUDA call failed."""
    dev = torch.device(device) if device is not None else (
        stream.device if stream is not None else _current_device())
    with _on_device(dev):
        site = int(lib.mimo_attn_checked_site(_stream(stream, dev)))
    if site < 0:
        raise MimoAttnError(MIMO_ERR_CUDA, lib.mimo_attn_last_error().decode())
    return site


def mimo_attn_checked_selftest(stream=None, device=None):
    """Checked build only: launch the one-thread kernel whose row check fails
    without touching memory (see include/mimo_attn.h)."""
    dev = torch.device(device) if device is not None else (
        stream.device if stream is not None else _current_device())
    with _on_device(dev):
        _check(lib.mimo_attn_checked_selftest(_stream(stream, dev)))


def default_scale(dqk=192):
    return 1.0 / math.sqrt(dqk)


def mimo_attn_decode_noalloc(q, k_cache, v_cache, seqlens, window, sinks, out, lse=None,
                             softmax_scale=None, v_scale=1.0, stream=None):
    """Decode through the entry point that allocates nothing (see include/mimo_attn.h).

    The caller passes preallocated ``out`` [B,Hq,128] and optional ``lse`` [B,Hq].
    """
    B, hq, dqk = q.shape
    C, hkv = k_cache.shape[1], k_cache.shape[2]
    _decode_shapes(q, k_cache, v_cache, seqlens, sinks, out, lse)
    dev = q.device
    _same_device(dev, k_cache=k_cache, v_cache=v_cache, seqlens=seqlens, sinks=sinks, out=out,
                 lse=lse)
    dims = make_dims(hq, hkv, dqk, v_cache.shape[3], softmax_scale, v_scale, out.dtype)
    with _on_device(dev):
        _check(lib.mimo_attn_decode_noalloc(ctypes.byref(dims), _ptr(q, "q", _BF16),
                                            _ptr(k_cache, "k_cache", _BF16),
                                            _ptr(v_cache, "v_cache", _BF16),
                                            _ptr(seqlens, "seqlens", _I32), B, C, int(window),
                                            _ptr(sinks, "sinks", _F32), _ptr(out, "out", _OUT),
                                            _ptr(lse, "lse", _F32), _stream(stream, dev)))
    return out, lse
