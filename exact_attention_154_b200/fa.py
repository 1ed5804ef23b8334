"""Python binding of ``libfa_sm100.so`` (the C ABI in ``include/fa.h``).

Argument marshalling only: torch supplies device memory and the current CUDA
stream; every step of the attention forward runs in the library's kernel.
There is no fallback: if the library is missing or the device is not an
sm_100 GPU, the calls raise.
"""
from __future__ import annotations

import ctypes
import functools
import math
import os
import threading

import torch

from .synth import BF16, FP16

_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libfa_sm100.so")
_lock = threading.Lock()
_lib = None

FA_OK = 0
FA_ERR_ARG, FA_ERR_ALIGN, FA_ERR_HEADDIM, FA_ERR_DTYPE = -1, -2, -3, -4
FA_ERR_UNSUPPORTED, FA_ERR_CUDA, FA_ERR_TIMEOUT, FA_ERR_DEVICE = -5, -6, -7, -8
FA_ERR_SEQLENS, FA_ERR_POSITIONS = -9, -10

FA_FP32 = 3
ROPE_SCALING = {"none": 0, "linear": 1, "ntk": 2, "yarn": 3}
NORM_ROPE_PARTS = 592

#: every function the C header declares, with (restype, argtypes)
_VP, _FP, _I, _F = ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int, ctypes.c_float
SIGNATURES = {
    "fa_fwd": (_I, [_VP, _VP, _VP, _VP, _FP, _I, _I, _I, _I, _F, _I, _I, _VP]),
    "fa_fwd_qkvpacked": (_I, [_VP, _VP, _FP, _I, _I, _I, _I, _F, _I, _F, _I, _VP]),
    "fa_fwd_ext": (_I, [_VP, _VP, _VP, _VP, _FP, _I, _I, _I, _I, _F, _I, _I, _I, _FP, _I, _VP]),
    "fa_fwd_qkvpacked_ext": (_I, [_VP, _VP, _FP, _I, _I, _I, _I, _F, _I, _F, _I, _I, _FP, _I,
                                  _VP]),
    "fa_fwd_fp8": (_I, [_VP, _VP, _VP, _VP, _FP, _I, _I, _I, _I, _F, _F, _F, _F, _I, _VP]),
    "fa_fwd_varlen": (_I, [_VP, _VP, _VP, _VP, _FP, _VP, _I, _I, _I, _I, _I, _F, _I, _I, _I, _FP,
                           _I, _VP]),
    "fa_bwd": (_I, [_VP, _VP, _VP, _VP, _FP, _VP, _VP, _VP, _VP, _FP, _I, _I, _I, _I, _F, _I, _I,
                    _VP]),
    "fa_bwd_noalloc": (_I, [_VP, _VP, _VP, _VP, _FP, _VP, _VP, _VP, _VP, _I, _I, _I, _I, _F, _I,
                            _I, _VP]),
    "fa_fwd_sinks": (_I, [_VP, _VP, _VP, _VP, _FP, _VP, _VP, _VP] + [_I] * 7 + [_F, _I, _VP]),
    "fa_bwd_sinks": (_I, [_VP, _VP, _VP, _VP, _FP] + [_VP] * 7 + [_FP] + [_I] * 7 + [_F, _I, _VP]),
    "fa_bwd_sinks_workspace": (ctypes.c_longlong, [_I] * 7),
    "fa_decode_sinks": (_I, [_VP, _VP, _VP, _VP, _FP, _VP, _VP, _VP] + [_I] * 7 + [_F, _I, _VP]),
    "fa_qk_norm_rope": (_I, [_VP] * 11 + [_I, _VP, _VP, _I, _F] + [_I] * 8 + [_VP]),
    "fa_qk_norm_rope_bwd": (_I, [_VP] * 15 + [_I, _VP, _VP, _I, _F, _FP] + [_I] * 8 + [_VP]),
    "fa_rope_table": (_I, [_FP, _FP, _I, _I, ctypes.c_double, _I, ctypes.c_double, _I, _VP]),
    "fa_strerror": (ctypes.c_char_p, [_I]),
    "fa_device_status": (_I, [_I, ctypes.POINTER(ctypes.c_uint)]),
    "fa_debug_watchdog_selftest": (_I, [ctypes.c_ulonglong, _VP]),
    "fa_launch_ctas": (_I, [_I, _I, _I, _I, _I]),
    "fa_debug_exp2_poly": (_I, [_VP, _VP, _I, _VP]),
    "fa_debug_set_wait_limit": (_I, [ctypes.c_ulonglong]),
    "fa_version": (_I, []),
}


class FaError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(f"{what}: {strerror(status)} ({status})")
        self.status = status


def lib_path() -> str:
    return _LIB_PATH


def load():
    """Load the shared library (raises if it has not been built)."""
    global _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(_LIB_PATH):
                raise RuntimeError(
                    f"{_LIB_PATH} is missing: build it with "
                    "`python -c 'import __graft_entry__ as g; g.build()'`")
            lib = ctypes.CDLL(_LIB_PATH)
            for name, (res, args) in SIGNATURES.items():
                fn = getattr(lib, name)
                fn.restype = res
                fn.argtypes = args
            _lib = lib
    return _lib


def strerror(status: int) -> str:
    return load().fa_strerror(int(status)).decode()


def version() -> int:
    return int(load().fa_version())


_DT = {torch.float16: FP16, torch.bfloat16: BF16}


def _stream_ptr(t: torch.Tensor):
    return ctypes.c_void_p(torch.cuda.current_stream(t.device).cuda_stream)


def same_device(named) -> torch.device:
    """The one device every ``(name, tensor)`` pair lives on; raises if they differ.

    The library resolves its per-device state (SM count, kernel attributes, the
    backward's scratch array) from the *current* device, so every call runs
    with the tensors' device made current (see :func:`_on`)."""
    dev = None
    for name, t in named:
        if dev is None:
            dev = t.device
        elif t.device != dev:
            raise ValueError(f"{name} is on {t.device}, expected {dev}")
    return dev


def _on(dev: torch.device):
    """Context that makes ``dev`` the current CUDA device for one library call."""
    return torch.cuda.device(dev)


def _check_tensor(t: torch.Tensor, name: str):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype not in _DT:
        raise ValueError(f"{name} must be float16 or bfloat16")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _window(window) -> tuple[int, int]:
    left, right = (int(window[0]), int(window[1]))
    return left, right


def _slopes(alibi_slopes, H: int, dev: torch.device):
    """The ``[H]`` fp32 slope tensor on ``dev`` (or None) and its pointer."""
    if alibi_slopes is None:
        return None, None
    if not isinstance(alibi_slopes, torch.Tensor):
        alibi_slopes = torch.as_tensor(alibi_slopes, dtype=torch.float32)
    if alibi_slopes.shape != (H,) or alibi_slopes.dtype != torch.float32:
        raise ValueError("alibi_slopes must be a float32 tensor of shape [H]")
    alibi_slopes = alibi_slopes.to(dev).contiguous()
    return alibi_slopes, alibi_slopes.data_ptr()


def fwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, scale: float | None = None,
        causal: bool = False, out: torch.Tensor | None = None,
        lse: torch.Tensor | None = None, return_lse: bool = True,
        window_size=(-1, -1), alibi_slopes=None):
    """Attention forward on ``[B, H, N, d]`` tensors (``[B, N, d]`` is taken as H=1).

    Returns ``(O, LSE)`` (``LSE`` is ``[B, H, N]`` fp32, or None when
    ``return_lse`` is False).  ``scale=None`` means ``1/sqrt(d)``.
    ``window_size=(left, right)``: key j visible from query i iff
    ``i - left <= j <= i + right`` (-1: unbounded).  ``alibi_slopes``: ``[H]``
    fp32; the scaled score gets ``-slope[h] * |i - j|``.
    """
    for name, t in (("q", q), ("k", k), ("v", v)):
        _check_tensor(t, name)
    if not (q.shape == k.shape == v.shape) or q.dtype != k.dtype or q.dtype != v.dtype:
        raise ValueError("q, k, v must share shape and dtype")
    if q.dim() == 3:
        B, N, d = q.shape
        H = 1
    elif q.dim() == 4:
        B, H, N, d = q.shape
    else:
        raise ValueError("expected [B, H, N, d] or [B, N, d]")
    if out is None:
        out = torch.empty_like(q)
    else:
        _check_tensor(out, "out")
        if out.shape != q.shape or out.dtype != q.dtype:
            raise ValueError("out must match q")
    lse_ptr = None
    if return_lse:
        if lse is None:
            lse = torch.empty((B, H, N), device=q.device, dtype=torch.float32)
        elif lse.shape != (B, H, N) or lse.dtype != torch.float32 or not lse.is_contiguous():
            raise ValueError("lse must be a contiguous [B, H, N] float32 tensor")
        lse_ptr = lse.data_ptr()
    else:
        lse = None
    dev = same_device([("q", q), ("k", k), ("v", v), ("out", out)] +
                      ([("lse", lse)] if lse is not None else []))
    left, right = _window(window_size)
    slopes, slopes_ptr = _slopes(alibi_slopes, H, dev)
    with _on(dev):
        rc = load().fa_fwd_ext(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
                               lse_ptr, B, H, N, d, 0.0 if scale is None else float(scale),
                               int(bool(causal)), left, right, slopes_ptr, _DT[q.dtype],
                               _stream_ptr(q))
    if rc != FA_OK:
        raise FaError(rc, "fa_fwd_ext")
    return out, lse


def fwd_qkvpacked(qkv: torch.Tensor, dropout_p: float = 0.0, softmax_scale: float | None = None,
                  causal: bool = False, out: torch.Tensor | None = None,
                  return_lse: bool = True, window_size=(-1, -1), alibi_slopes=None):
    """Packed forward: ``qkv`` is ``[B, N, 3, H, d]``; returns ``(O [B, N, H, d], LSE [B, H, N])``.

    ``window_size`` and ``alibi_slopes`` as :func:`fwd`."""
    _check_tensor(qkv, "qkv")
    if qkv.dim() != 5 or qkv.shape[2] != 3:
        raise ValueError("qkv must be [B, N, 3, H, d]")
    B, N, _, H, d = qkv.shape
    if out is None:
        out = torch.empty((B, N, H, d), device=qkv.device, dtype=qkv.dtype)
    else:
        _check_tensor(out, "out")
    if out.shape != (B, N, H, d) or out.dtype != qkv.dtype:
        raise ValueError("out must be [B, N, H, d] in qkv's dtype")
    lse = torch.empty((B, H, N), device=qkv.device, dtype=torch.float32) if return_lse else None
    dev = same_device([("qkv", qkv), ("out", out)])
    left, right = _window(window_size)
    slopes, slopes_ptr = _slopes(alibi_slopes, H, dev)
    with _on(dev):
        rc = load().fa_fwd_qkvpacked_ext(
            qkv.data_ptr(), out.data_ptr(), None if lse is None else lse.data_ptr(), B, N, H, d,
            0.0 if softmax_scale is None else float(softmax_scale), int(bool(causal)),
            float(dropout_p), left, right, slopes_ptr, _DT[qkv.dtype], _stream_ptr(qkv))
    if rc != FA_OK:
        raise FaError(rc, "fa_fwd_qkvpacked_ext")
    return out, lse


def fwd_fp8(q8: torch.Tensor, k8: torch.Tensor, v8: torch.Tensor, descale_q: float,
            descale_k: float, descale_v: float, scale: float | None = None,
            causal: bool = False, return_lse: bool = True):
    """Forward on fp8 e4m3 ``[B, H, N, d]`` tensors (torch.float8_e4m3fn, or
    uint8 holding the codes) with per-tensor dequantisation factors: the real
    operands are ``descale_x * x``.  Returns ``(O bf16 [B, H, N, d], LSE)``."""
    for name, t in (("q8", q8), ("k8", k8), ("v8", v8)):
        if not isinstance(t, torch.Tensor) or not t.is_cuda:
            raise ValueError(f"{name} must be a CUDA tensor")
        if t.dtype not in (torch.float8_e4m3fn, torch.uint8) or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous float8_e4m3fn (or uint8) tensor")
    if not (q8.shape == k8.shape == v8.shape) or q8.dim() != 4:
        raise ValueError("q8, k8, v8 must share one [B, H, N, d] shape")
    B, H, N, d = q8.shape
    dev = same_device([("q8", q8), ("k8", k8), ("v8", v8)])
    out = torch.empty((B, H, N, d), device=dev, dtype=torch.bfloat16)
    lse = torch.empty((B, H, N), device=dev, dtype=torch.float32) if return_lse else None
    with _on(dev):
        rc = load().fa_fwd_fp8(q8.data_ptr(), k8.data_ptr(), v8.data_ptr(), out.data_ptr(),
                               None if lse is None else lse.data_ptr(), B, H, N, d,
                               0.0 if scale is None else float(scale), float(descale_q),
                               float(descale_k), float(descale_v), int(bool(causal)),
                               _stream_ptr(q8))
    if rc != FA_OK:
        raise FaError(rc, "fa_fwd_fp8")
    return out, lse


def fwd_varlen(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cu_seqlens: torch.Tensor,
               max_seqlen: int, scale: float | None = None, causal: bool = False,
               window_size=(-1, -1), alibi_slopes=None, return_lse: bool = True):
    """Forward over sequences packed back to back: ``q, k, v`` are
    ``[total, H, d]``, sequence b holds rows ``cu_seqlens[b] .. cu_seqlens[b+1]-1``
    (``cu_seqlens``: int32 ``[batch + 1]`` on the same device).  Returns
    ``(O [total, H, d], LSE [H, total])``.  Masks as :func:`fwd`, per sequence."""
    for name, t in (("q", q), ("k", k), ("v", v)):
        _check_tensor(t, name)
    if not (q.shape == k.shape == v.shape) or q.dim() != 3 or len({q.dtype, k.dtype, v.dtype}) != 1:
        raise ValueError("q, k, v must share one [total, H, d] shape and dtype")
    if (not isinstance(cu_seqlens, torch.Tensor) or cu_seqlens.dtype != torch.int32
            or cu_seqlens.dim() != 1 or cu_seqlens.numel() < 2 or not cu_seqlens.is_contiguous()):
        raise ValueError("cu_seqlens must be a contiguous int32 tensor of batch + 1 offsets")
    total, H, d = q.shape
    batch = cu_seqlens.numel() - 1
    dev = same_device([("q", q), ("k", k), ("v", v), ("cu_seqlens", cu_seqlens)])
    out = torch.empty_like(q)
    lse = torch.empty((H, total), device=dev, dtype=torch.float32) if return_lse else None
    left, right = _window(window_size)
    slopes, slopes_ptr = _slopes(alibi_slopes, H, dev)
    with _on(dev):
        rc = load().fa_fwd_varlen(
            q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
            None if lse is None else lse.data_ptr(), cu_seqlens.data_ptr(), batch,
            int(max_seqlen), total, H, d, 0.0 if scale is None else float(scale),
            int(bool(causal)), left, right, slopes_ptr, _DT[q.dtype], _stream_ptr(q))
    if rc != FA_OK:
        raise FaError(rc, "fa_fwd_varlen")
    return out, lse


def bwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, o: torch.Tensor, lse: torch.Tensor,
        dout: torch.Tensor, scale: float | None = None, causal: bool = False):
    """Gradient of :func:`fwd`: returns ``(dQ, dK, dV)`` for an upstream ``dout``.

    ``o`` and ``lse`` are the outputs of :func:`fwd` on the same ``q, k, v``,
    ``scale`` and ``causal``; all tensors ``[B, H, N, d]`` (``lse`` ``[B, H, N]``
    fp32).  The fp32 row-statistic workspace is allocated here.
    """
    for name, t in (("q", q), ("k", k), ("v", v), ("o", o), ("dout", dout)):
        _check_tensor(t, name)
    if not (q.shape == k.shape == v.shape == o.shape == dout.shape) or q.dim() != 4:
        raise ValueError("q, k, v, o, dout must share one [B, H, N, d] shape")
    if len({t.dtype for t in (q, k, v, o, dout)}) != 1:
        raise ValueError("q, k, v, o, dout must share one dtype")
    B, H, N, d = q.shape
    if lse.shape != (B, H, N) or lse.dtype != torch.float32 or not lse.is_contiguous():
        raise ValueError("lse must be a contiguous [B, H, N] float32 tensor")
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    dev = same_device([("q", q), ("k", k), ("v", v), ("o", o), ("lse", lse), ("dout", dout)])
    work = torch.empty((B, H, N), device=q.device, dtype=torch.float32)
    with _on(dev):
        rc = load().fa_bwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(),
                           dout.data_ptr(), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(),
                           work.data_ptr(), B, H, N, d, 0.0 if scale is None else float(scale),
                           int(bool(causal)), _DT[q.dtype], _stream_ptr(q))
    if rc != FA_OK:
        raise FaError(rc, "fa_bwd")
    return dq, dk, dv


def bwd_noalloc(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, o: torch.Tensor,
                lse: torch.Tensor, dout: torch.Tensor, scale: float | None = None,
                causal: bool = False):
    """:func:`bwd` through ``fa_bwd_noalloc``: the row statistic lives in the
    library's own device array instead of a workspace tensor."""
    for name, t in (("q", q), ("k", k), ("v", v), ("o", o), ("dout", dout)):
        _check_tensor(t, name)
    if not (q.shape == k.shape == v.shape == o.shape == dout.shape) or q.dim() != 4:
        raise ValueError("q, k, v, o, dout must share one [B, H, N, d] shape")
    if len({t.dtype for t in (q, k, v, o, dout)}) != 1:
        raise ValueError("q, k, v, o, dout must share one dtype")
    B, H, N, d = q.shape
    if lse.shape != (B, H, N) or lse.dtype != torch.float32 or not lse.is_contiguous():
        raise ValueError("lse must be a contiguous [B, H, N] float32 tensor")
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    dev = same_device([("q", q), ("k", k), ("v", v), ("o", o), ("lse", lse), ("dout", dout)])
    with _on(dev):
        rc = load().fa_bwd_noalloc(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(),
                                   lse.data_ptr(), dout.data_ptr(), dq.data_ptr(), dk.data_ptr(),
                                   dv.data_ptr(), B, H, N, d,
                                   0.0 if scale is None else float(scale), int(bool(causal)),
                                   _DT[q.dtype], _stream_ptr(q))
    if rc != FA_OK:
        raise FaError(rc, "fa_bwd_noalloc")
    return dq, dk, dv


def _check_rows(t: torch.Tensor, name: str, dtype=None):
    """A 16-bit CUDA tensor [B, H, N, d] whose rows are adjacent elements."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype is not dtype and (t.dtype not in _DT or dtype is not None):
        raise ValueError(f"{name} must be float16 or bfloat16, one type for all operands")
    if t.dim() != 4 or t.stride(3) != 1:
        raise ValueError(f"{name} must be [B, H, N, d] with adjacent elements in a row")


@functools.lru_cache(maxsize=256)
def _stride_array(b, h, n):
    return (ctypes.c_longlong * 3)(b, h, n)


def _strides(t: torch.Tensor):
    """The (batch, head, row) strides argument of the C ABI; None when contiguous."""
    return None if t.is_contiguous() else _stride_array(*t.stride()[:3])


def _launch(what: str, names: str, tensors, args):
    """Calls entry point ``what`` with ``args`` and the current stream of the first
    of ``tensors``, with its device current.  The others (or None; ``names`` are
    theirs) must live on that device.  Raises what the library refuses."""
    index = tensors[0].get_device()
    for t in tensors:
        if t is not None and t.get_device() != index:
            same_device((n, x) for n, x in zip(names.split(), tensors) if x is not None)
    fn = getattr(_lib or load(), what)
    if torch._C._cuda_getDevice() == index:
        rc = fn(*args, torch._C._cuda_getCurrentRawStream(index))
    else:
        with _on(tensors[0].device):
            rc = fn(*args, torch._C._cuda_getCurrentRawStream(index))
    if rc != FA_OK:
        raise FaError(rc, what)


def _new_like(t: torch.Tensor):
    """A new contiguous tensor of ``t``'s shape, type and device."""
    return torch.empty_like(t, memory_format=torch.contiguous_format)


def _check_out(t: torch.Tensor, name: str, like: torch.Tensor):
    """A given output: its input's shape and type, rows that do not overlap."""
    _check_rows(t, name, like.dtype)
    if t.shape != like.shape or not _fresh_rows(t):
        raise ValueError(f"{name} must have its input's shape and rows that do not overlap")


def _fresh_rows(t: torch.Tensor):
    """Whether the rows of [B, H, N, d] tensor ``t`` surely do not overlap: its
    dimensions, ordered by stride, each step over the one before."""
    need = 0
    for size, stride in sorted(((n, s) for n, s in zip(t.shape, t.stride()) if n > 1),
                               key=lambda x: x[1]):
        if stride <= need:
            return False
        need += (size - 1) * stride
    return True


def _fits(t, dtype, shape) -> bool:
    """Whether ``t`` is a contiguous tensor of this type and shape."""
    return isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape \
        and t.is_contiguous()


def _table(cos, sin, positions, B, N):
    """Checks of the cos / sin table and the positions; (max_pos, rot)."""
    shape = cos.shape if isinstance(cos, torch.Tensor) else ()
    if len(shape) != 2 or not _fits(cos, torch.float32, shape) \
            or not _fits(sin, torch.float32, shape):
        raise ValueError("cos and sin must be contiguous float32 [max_pos, rot / 2] tensors")
    if positions is not None and not _fits(positions, torch.int32, (B, N)):
        raise ValueError("positions must be a contiguous int32 [B, N] tensor")
    return shape[0], 2 * shape[1]


def _weights(q_weight, k_weight, d, dtype):
    """Checks of the norm weights; the type code the library is told."""
    first = k_weight if q_weight is None else q_weight
    if first is None:
        return _DT[dtype]
    wt = first.dtype if isinstance(first, torch.Tensor) else None
    if wt not in (dtype, torch.float32) or not _fits(first, wt, (d,)) \
            or (k_weight is not None and k_weight is not first and not _fits(k_weight, wt, (d,))):
        raise ValueError("q_weight and k_weight must be contiguous [d] tensors of the operands' "
                         "type or float32, both of one type")
    return FA_FP32 if wt is torch.float32 else _DT[dtype]


def _ptr(t):
    return None if t is None else t.data_ptr()


def _check_qkv(q, k, v):
    """Checks of [B, H, N, d] queries against [B, Hk, N, d] keys and values."""
    _check_rows(q, "q")
    _check_rows(k, "k", q.dtype)
    _check_rows(v, "v", q.dtype)
    B, H, N, d = q.shape
    if k.shape != v.shape or k.shape != (B, k.shape[1], N, d) or k.shape[1] < 1 \
            or H % k.shape[1] != 0:
        raise ValueError("k and v must be [B, Hk, N, d] with q's B, N and d, H a multiple of Hk")
    return B, H, k.shape[1], N, d


def _check_lse(lse, shape):
    if not isinstance(lse, torch.Tensor) or lse.shape != shape or lse.dtype != torch.float32 \
            or not lse.is_contiguous():
        raise ValueError(f"lse must be a contiguous {list(shape)} float32 tensor")


def fwd_sinks(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, window: int, sinks: int,
              scale: float | None = None, out: torch.Tensor | None = None,
              lse: torch.Tensor | None = None, return_lse: bool = True):
    """Causal attention over a sliding window plus the first ``sinks`` tokens,
    which stay visible from every later query: key j is visible from query i iff
    ``j <= i and (i - j <= window or j < sinks)`` (``window=-1``: plain causal).

    ``q`` is ``[B, H, N, d]``, ``k`` and ``v`` ``[B, Hk, N, d]`` (each key head
    shared by ``H / Hk`` query heads), of any strides with adjacent row elements.
    Returns ``(O [B, H, N, d], LSE [B, H, N])``, contiguous; LSE is None when
    ``return_lse`` is False."""
    B, H, Hk, N, d = _check_qkv(q, k, v)
    if out is None:
        out = _new_like(q)
    else:
        _check_tensor(out, "out")
        if out.shape != q.shape or out.dtype != q.dtype:
            raise ValueError("out must match q")
    if not return_lse:
        lse = None
    elif lse is None:
        lse = torch.empty((B, H, N), device=q.device, dtype=torch.float32)
    else:
        _check_lse(lse, (B, H, N))
    _launch("fa_fwd_sinks", "q k v out lse", (q, k, v, out, lse),
            (q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), _ptr(lse), _strides(q),
             _strides(k), _strides(v), B, H, Hk, N, d, int(window), int(sinks),
             0.0 if scale is None else float(scale), _DT[q.dtype]))
    return out, lse


def bwd_sinks(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, o: torch.Tensor,
              lse: torch.Tensor, dout: torch.Tensor, window: int, sinks: int,
              scale: float | None = None):
    """Gradient of :func:`fwd_sinks` for an upstream gradient ``dout`` of its O:
    ``(dq [B, H, N, d], dk, dv [B, Hk, N, d])``, contiguous; ``dk`` and ``dv``
    are summed over the query heads that share a key head.  ``o``, ``lse``: the
    forward's results; ``o`` and ``dout`` contiguous.  d is 64 or 128."""
    B, H, Hk, N, d = _check_qkv(q, k, v)
    for name, t in (("o", o), ("dout", dout)):
        _check_tensor(t, name)
        if t.shape != q.shape or t.dtype != q.dtype:
            raise ValueError(f"{name} must match q")
    _check_lse(lse, (B, H, N))
    floats = load().fa_bwd_sinks_workspace(B, H, Hk, N, d, int(window), int(sinks))
    if floats < 0:
        raise FaError(int(floats), "fa_bwd_sinks_workspace")
    dq, dk, dv = _new_like(q), _new_like(k), _new_like(v)
    ws = lse.new_empty((floats,))
    _launch("fa_bwd_sinks", "q k v o lse dout", (q, k, v, o, lse, dout),
            (q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(),
             dout.data_ptr(), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), _strides(q),
             _strides(k), _strides(v), ws.data_ptr(), B, H, Hk, N, d, int(window), int(sinks),
             0.0 if scale is None else float(scale), _DT[q.dtype]))
    return dq, dk, dv


def decode_sinks(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, seqlens: torch.Tensor,
                 window: int, sinks: int, scale: float | None = None,
                 out: torch.Tensor | None = None, return_lse: bool = True):
    """:func:`fwd_sinks` one token at a time: ``q`` ``[B, H, d]`` holds each
    sequence's newest query, ``k`` and ``v`` ``[B, Hk, S, d]`` (any strides with
    adjacent row elements) its cached keys and values, of which the first
    ``seqlens[b]`` (int32 ``[B]``, the newest token included) are in use.
    Returns ``(O [B, H, d], LSE [B, H])``; a length of 0 gives O = 0 and LSE =
    -inf.  Cache rows that are not visible may hold anything."""
    _check_tensor(q, "q")
    if q.dim() != 3:
        raise ValueError("q must be [B, H, d]")
    B, H, d = q.shape
    _check_rows(k, "k", q.dtype)
    _check_rows(v, "v", q.dtype)
    Hk, S = k.shape[1], k.shape[2]
    if k.shape != v.shape or k.shape != (B, Hk, S, d) or Hk < 1 or H % Hk != 0:
        raise ValueError("k and v must be [B, Hk, S, d] with q's B and d, H a multiple of Hk")
    if not isinstance(seqlens, torch.Tensor) or seqlens.dtype != torch.int32 \
            or seqlens.shape != (B,) or not seqlens.is_contiguous():
        raise ValueError("seqlens must be a contiguous int32 [B] tensor")
    if out is None:
        out = torch.empty_like(q)
    else:
        _check_tensor(out, "out")
        if out.shape != q.shape or out.dtype != q.dtype:
            raise ValueError("out must match q")
    lse = q.new_empty((B, H), dtype=torch.float32) if return_lse else None
    _launch("fa_decode_sinks", "q k v seqlens out", (q, k, v, seqlens, out),
            (q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), _ptr(lse),
             seqlens.data_ptr(), _strides(k), _strides(v), B, H, Hk, S, d, int(window), int(sinks),
             0.0 if scale is None else float(scale), _DT[q.dtype]))
    return out, lse


def rope_table(max_pos: int, rot: int, base: float = 10000.0, scaling: str = "none",
               factor: float = 1.0, original_max_pos: int = 0, device="cuda"):
    """``(cos, sin)``, each ``[max_pos, rot / 2]`` fp32: the table of
    :func:`qk_norm_rope` for angles ``p * base ** (-2 i / rot)``.

    ``scaling`` for contexts longer than trained on: ``"linear"`` (frequencies
    over ``factor``), ``"ntk"`` (a larger base), ``"yarn"`` (slow pairs
    interpolated, fast ones kept; needs ``original_max_pos``)."""
    if scaling not in ROPE_SCALING:
        raise ValueError(f"scaling must be one of {sorted(ROPE_SCALING)}")
    dev = torch.device(device)
    if dev.type != "cuda":
        raise ValueError("device must be a CUDA device")
    if max_pos < 1 or rot < 2:
        raise ValueError("max_pos and rot must be positive")
    cos = torch.empty((max_pos, rot // 2), device=dev, dtype=torch.float32)
    sin = torch.empty_like(cos)
    _launch("fa_rope_table", "cos", (cos,),
            (cos.data_ptr(), sin.data_ptr(), max_pos, rot, float(base), ROPE_SCALING[scaling],
             float(factor), int(original_max_pos)))
    return cos, sin


def qk_norm_rope(q: torch.Tensor, k: torch.Tensor, cos: torch.Tensor, sin: torch.Tensor,
                 positions: torch.Tensor | None = None, q_weight: torch.Tensor | None = None,
                 k_weight: torch.Tensor | None = None, eps: float = 1e-6,
                 interleaved: bool = False, q_out: torch.Tensor | None = None,
                 k_out: torch.Tensor | None = None):
    """RMS norm of every head's query and key and the rotation by position.

    ``q`` is ``[B, H, N, d]``, ``k`` ``[B, Hk, N, d]``, of any strides with
    adjacent row elements (views of a packed projection, ``transpose(1, 2)`` of
    ``[B, N, H, d]``).  ``cos``, ``sin``: ``[max_pos, rot / 2]`` fp32
    (:func:`rope_table`); ``positions`` int32 ``[B, N]`` (None: the row index).
    ``q_weight``, ``k_weight``: ``[d]``, or None to leave that operand
    unnormalised.  Returns ``(q_out, k_out)``, contiguous unless given; they
    may be ``q`` and ``k`` themselves."""
    _check_rows(q, "q")
    _check_rows(k, "k", q.dtype)
    B, H, N, d = q.shape
    Hk = k.shape[1]
    if k.shape != (B, Hk, N, d):
        raise ValueError("k must be [B, Hk, N, d] with q's B, N and d")
    max_pos, rot = _table(cos, sin, positions, B, N)
    wt = _weights(q_weight, k_weight, d, q.dtype)
    qo = ko = None  # strides of given outputs
    if q_out is None:
        q_out = _new_like(q)
    else:
        _check_out(q_out, "q_out", q)
        qo = _strides(q_out)
    if k_out is None:
        k_out = _new_like(k)
    else:
        _check_out(k_out, "k_out", k)
        ko = _strides(k_out)
    _launch("fa_qk_norm_rope", "q k cos sin positions q_weight k_weight q_out k_out",
            (q, k, cos, sin, positions, q_weight, k_weight, q_out, k_out),
            (q.data_ptr(), k.data_ptr(), q_out.data_ptr(), k_out.data_ptr(), _strides(q),
             _strides(k), qo, ko, cos.data_ptr(), sin.data_ptr(),
             _ptr(positions), max_pos, _ptr(q_weight), _ptr(k_weight), wt, float(eps), B, H, Hk, N,
             d, rot, int(bool(interleaved)), _DT[q.dtype]))
    return q_out, k_out


def qk_norm_rope_bwd(dq_out: torch.Tensor, dk_out: torch.Tensor, q: torch.Tensor, k: torch.Tensor,
                     cos: torch.Tensor, sin: torch.Tensor, positions: torch.Tensor | None = None,
                     q_weight: torch.Tensor | None = None, k_weight: torch.Tensor | None = None,
                     eps: float = 1e-6, interleaved: bool = False):
    """Gradient of :func:`qk_norm_rope` for gradients ``dq_out``, ``dk_out`` of
    its results; ``q``, ``k`` and the rest are the forward's arguments.
    Returns ``(dq, dk, dq_weight, dk_weight)``, the first two contiguous, the
    last two None where the weight is None."""
    _check_rows(q, "q")
    B, H, N, d = q.shape
    Hk = k.shape[1] if isinstance(k, torch.Tensor) and k.dim() == 4 else 0
    for name, t, shape in (("k", k, (B, Hk, N, d)), ("dq_out", dq_out, q.shape),
                           ("dk_out", dk_out, (B, Hk, N, d))):
        _check_rows(t, name, q.dtype)
        if t.shape != shape:
            raise ValueError(f"{name} does not match q and k")
    max_pos, rot = _table(cos, sin, positions, B, N)
    wt = _weights(q_weight, k_weight, d, q.dtype)
    dq, dk = _new_like(q), _new_like(k)
    dqw = None if q_weight is None else torch.empty_like(q_weight)
    dkw = None if k_weight is None else torch.empty_like(k_weight)
    ws = cos.new_empty((NORM_ROPE_PARTS, d))
    _launch("fa_qk_norm_rope_bwd", "q k dq_out dk_out cos sin positions q_weight k_weight",
            (q, k, dq_out, dk_out, cos, sin, positions, q_weight, k_weight),
            (dq_out.data_ptr(), dk_out.data_ptr(), q.data_ptr(), k.data_ptr(), dq.data_ptr(),
             dk.data_ptr(), _ptr(dqw), _ptr(dkw), _strides(dq_out), _strides(dk_out), _strides(q),
             _strides(k), cos.data_ptr(), sin.data_ptr(), _ptr(positions), max_pos, _ptr(q_weight),
             _ptr(k_weight), wt, float(eps), ws.data_ptr(), B, H, Hk, N, d, rot,
             int(bool(interleaved)), _DT[q.dtype]))
    return dq, dk, dqw, dkw


def device_status(clear: bool = True):
    """(status, detail) of the current device's watchdog word; synchronises."""
    detail = ctypes.c_uint(0)
    rc = load().fa_device_status(int(bool(clear)), ctypes.byref(detail))
    return int(rc), int(detail.value)


def watchdog_selftest(limit_ns: int = 20_000_000):
    """Run the bounded-wait self test kernel on the current stream."""
    rc = load().fa_debug_watchdog_selftest(int(limit_ns),
                                           ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
    if rc != FA_OK:
        raise FaError(rc, "fa_debug_watchdog_selftest")


def set_wait_limit(limit_ns: int = 0):
    """Bound (ns) of every mbarrier wait in the kernels launched next; 0
    restores the default.  A debug hook for testing the kernels' give-up path."""
    rc = load().fa_debug_set_wait_limit(int(limit_ns))
    if rc != FA_OK:
        raise FaError(rc, "fa_debug_set_wait_limit")


def exp2_poly(x: torch.Tensor) -> torch.Tensor:
    """The kernel's software exp2 applied to a float32 CUDA tensor (test hook)."""
    if not x.is_cuda or x.dtype != torch.float32 or not x.is_contiguous():
        raise ValueError("x must be a contiguous float32 CUDA tensor")
    y = torch.empty_like(x)
    rc = load().fa_debug_exp2_poly(x.data_ptr(), y.data_ptr(), x.numel(), _stream_ptr(x))
    if rc != FA_OK:
        raise FaError(rc, "fa_debug_exp2_poly")
    return y


def launch_ctas(B: int, H: int, N: int, d: int, causal: bool = False) -> int:
    return int(load().fa_launch_ctas(B, H, N, d, int(bool(causal))))


def default_scale(d: int) -> float:
    """The fp32 scale the library uses when none is given: 1/sqrt(d) rounded to fp32."""
    return float(torch.tensor(1.0 / math.sqrt(d), dtype=torch.float32))
