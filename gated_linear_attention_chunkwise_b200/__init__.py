"""DiG gated-linear-attention hot path on B200 -- thin Python binding.

Every function here only checks shapes/dtypes (for readable errors), picks the
caller's current CUDA stream and forwards raw device pointers to the C ABI of
`libdig_gla.so` (declared in include/dig_gla.h).  All computation happens in
the library's sm_100a kernels; there is no CPU or PyTorch fallback, and
importing this package fails if the library has not been built
(`python gated_linear_attention_chunkwise_b200/build.py`).

Names follow the C ABI: gla_fwd, gla_fwd_glogit, gla_fwd_f32, gla_bwd, gla_bwd_f32, gla_norm_fwd,
gla_norm_fwd_f32, srem_reorient, dwconv3x3, glr_fwd, glr_fwd_packed, glr_bwd, glr_bwd_packed, glr_step, rope,
qk_norm_rope, qk_norm_rope_bwd,
device_status (dig_gla_device_status), status_string (dig_gla_status_string).
"""
from __future__ import annotations

import ctypes
import math
import os

import torch

__all__ = ["gla_fwd", "gla_fwd_glogit", "gla_fwd_f32", "gla_bwd", "gla_bwd_f32", "gla_norm_fwd", "gla_norm_fwd_f32", "srem_reorient", "dwconv3x3",
           "glr_fwd", "glr_fwd_packed", "glr_bwd", "glr_bwd_packed", "glr_step", "rope", "qk_norm_rope", "qk_norm_rope_bwd",
           "rope_frequencies", "device_status", "status_string",
           "GlaError", "lib", "LIB_PATH", "DIR_L2R", "DIR_R2L", "DIR_T2B", "DIR_B2T"]

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libdig_gla.so")
if not os.path.exists(LIB_PATH):
    raise ImportError(f"{LIB_PATH} is missing: build it with `python gated_linear_attention_chunkwise_b200/build.py`"
                      " (nvcc, sm_100a). There is no fallback implementation.")

_lib = ctypes.CDLL(LIB_PATH)
_vp, _i, _u = ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p
_lib.gla_fwd.argtypes = [_vp, _vp, _vp, _vp] + [_i] * 7 + [_vp, _u]
_lib.gla_fwd_f32.argtypes = [_vp, _vp, _vp, _vp] + [_i] * 7 + [_vp, _u]
_lib.gla_bwd.argtypes = [_vp] * 5 + [_i] * 7 + [_vp] * 4 + [_u]
_lib.gla_bwd_f32.argtypes = [_vp] * 5 + [_i] * 7 + [_vp] * 4 + [_u]
_lib.gla_fwd_glogit.argtypes = [_vp] * 4 + [_i] * 7 + [ctypes.c_float, _vp, _u]
_lib.gla_norm_fwd.argtypes = [_vp] * 3 + [_i] * 7 + [ctypes.c_float, _vp, _u]
_lib.gla_norm_fwd_f32.argtypes = [_vp] * 3 + [_i] * 7 + [ctypes.c_float, _vp, _u]
_lib.srem_reorient.argtypes = [_vp, _i, _i, _i, _i, _i, _i, _i, _vp, _u]
_lib.dwconv3x3.argtypes = [_vp, _vp, _i, _i, _i, _i, _i, _vp, _u]
_i64, _f = ctypes.c_int64, ctypes.c_float
_lib.glr_fwd.argtypes = [_vp] * 3 + [_i] * 4 + [_i64] * 2 + [_i, _f, _i, _i] + [_vp] * 2 + [_u]
_lib.glr_fwd_packed.argtypes = [_vp] * 4 + [_i64] + [_i] * 2 + [_i64] * 2 + [_i, _f, _i, _i, _i] + [_vp] * 2 + [_u]
_lib.glr_bwd.argtypes = [_vp] * 6 + [_i] * 4 + [_i64] * 2 + [_i, _f, _i, _i] + [_vp] * 3 + [_u]
_lib.glr_bwd_packed.argtypes = [_vp] * 7 + [_i64] + [_i] * 2 + [_i64] * 2 + [_i, _f, _i, _i, _i] + [_vp] * 3 + [_u]
_lib.glr_step.argtypes = [_vp] * 4 + [_i] * 3 + [_i64] * 2 + [_f, _i, _i, _i] + [_vp] * 2 + [_u]
_lib.rope.argtypes = [_vp] * 3 + [_i] * 2 + [_vp, _i64] + [_i] * 4 + [_i64] * 2 + [_i] * 2 + [_f, _i] + [_vp, _i64] * 2 + [_u]
_lib.qk_norm_rope.argtypes = ([_vp] * 5 + [_i] * 2 + [_vp, _i64] + [_i] * 4 + [_i64] * 2 + [_i, _f, _f, _i] + [_vp, _i64] * 2 +
                              [_u])
_lib.qk_norm_rope_bwd.argtypes = ([_vp] * 7 + [_i] * 2 + [_vp, _i64] + [_i] * 4 + [_i64] * 4 + [_i, _f, _f, _i] +
                                  [_vp, _i64] * 2 + [_vp] * 2 + [_u])
_lib.dig_gla_device_status.argtypes = [_u]
_lib.dig_gla_status_string.argtypes = [_i]
_lib.dig_gla_status_string.restype = ctypes.c_char_p
_lib.dig_gla_release.argtypes = []
_lib.dig_gla_release.restype = None
_lib.dig_gla_test_skip_items.argtypes = [_i]
_lib.dig_gla_test_skip_items.restype = None
for _fn in (_lib.gla_fwd, _lib.gla_fwd_glogit, _lib.gla_fwd_f32, _lib.gla_bwd, _lib.gla_bwd_f32, _lib.gla_norm_fwd, _lib.gla_norm_fwd_f32,
            _lib.srem_reorient, _lib.dwconv3x3, _lib.glr_fwd, _lib.glr_fwd_packed, _lib.glr_bwd, _lib.glr_bwd_packed,
            _lib.glr_step, _lib.rope, _lib.qk_norm_rope, _lib.qk_norm_rope_bwd, _lib.dig_gla_device_status):
    _fn.restype = ctypes.c_int

DIR_L2R, DIR_R2L, DIR_T2B, DIR_B2T = 0, 1, 2, 3
_BF16, _F32 = 0, 1


def lib() -> ctypes.CDLL:
    """The loaded C library (for callers that pass raw pointers themselves)."""
    return _lib


class GlaError(RuntimeError):
    def __init__(self, fn: str, code: int):
        super().__init__(f"{fn} failed: {status_string(code)} ({code})")
        self.code = code


def status_string(code: int) -> str:
    return _lib.dig_gla_status_string(int(code)).decode()


def _check(fn: str, rc: int):
    if rc != 0:
        raise GlaError(fn, rc)


def _stream_handle(dev: torch.device, stream) -> int:
    if stream is None:
        stream = torch.cuda.current_stream(dev)
    return int(stream.cuda_stream) if hasattr(stream, "cuda_stream") else int(stream)


def _need(t: torch.Tensor, name: str, dtype: torch.dtype, dev: torch.device):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device != dev or t.device.type != "cuda":
        raise ValueError(f"{name} must be on {dev} (got {t.device})")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype} (got {t.dtype})")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _gla(fn_name: str, q, k, v, log_alpha, Hgrid, Wgrid, direction, out, stream, dtype):
    dev = q.device
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _need(t, n, dtype, dev)
    _need(log_alpha, "log_alpha", torch.float32, dev)
    if q.dim() != 4 or k.shape != q.shape or log_alpha.shape != q.shape or v.dim() != 4 or v.shape[:3] != q.shape[:3]:
        raise ValueError("expected q, k, log_alpha [B,T,H,dk] and v [B,T,H,dv]")
    B, T, H, dk = q.shape
    dv = v.shape[3]
    if T != Hgrid * Wgrid:
        raise ValueError(f"T={T} does not match the grid {Hgrid}x{Wgrid}")
    if out is None:
        out = torch.empty((B, T, H, dv), dtype=dtype, device=dev)
    else:
        _need(out, "out", dtype, dev)
        if tuple(out.shape) != (B, T, H, dv):
            raise ValueError("out must be [B,T,H,dv]")
    with torch.cuda.device(dev):
        rc = getattr(_lib, fn_name)(q.data_ptr(), k.data_ptr(), v.data_ptr(), log_alpha.data_ptr(), B, H, Hgrid,
                                    Wgrid, dk, dv, int(direction), out.data_ptr(), _stream_handle(dev, stream))
    _check(fn_name, rc)
    return out


def gla_fwd(q, k, v, log_alpha, Hgrid: int, Wgrid: int, direction: int, out=None, stream=None):
    """bf16 GLA forward (see include/dig_gla.h, gla_fwd).  Returns `out` [B,T,H,dv] bf16."""
    return _gla("gla_fwd", q, k, v, log_alpha, Hgrid, Wgrid, direction, out, stream, torch.bfloat16)


def gla_fwd_glogit(q, k, v, g, Hgrid: int, Wgrid: int, direction: int, gate_norm: float = 16.0, out=None,
                   stream=None):
    """bf16 GLA forward with bf16 gate logits g (log_alpha = logsigmoid(g) / gate_norm in
    the kernel; see include/dig_gla.h, gla_fwd_glogit).  Returns `out` [B,T,H,dv] bf16."""
    dev = q.device
    for t, n in ((q, "q"), (k, "k"), (v, "v"), (g, "g")):
        _need(t, n, torch.bfloat16, dev)
    if q.dim() != 4 or k.shape != q.shape or g.shape != q.shape or v.dim() != 4 or v.shape[:3] != q.shape[:3]:
        raise ValueError("expected q, k, g [B,T,H,dk] and v [B,T,H,dv]")
    B, T, H, dk = q.shape
    dv = v.shape[3]
    if T != Hgrid * Wgrid:
        raise ValueError(f"T={T} does not match the grid {Hgrid}x{Wgrid}")
    if out is None:
        out = torch.empty((B, T, H, dv), dtype=torch.bfloat16, device=dev)
    else:
        _need(out, "out", torch.bfloat16, dev)
    with torch.cuda.device(dev):
        rc = _lib.gla_fwd_glogit(q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(), B, H, Hgrid, Wgrid, dk, dv,
                                 int(direction), float(gate_norm), out.data_ptr(), _stream_handle(dev, stream))
    _check("gla_fwd_glogit", rc)
    return out


def gla_fwd_f32(q, k, v, log_alpha, Hgrid: int, Wgrid: int, direction: int, out=None, stream=None):
    """fp32 GLA forward (see include/dig_gla.h, gla_fwd_f32).  Returns `out` [B,T,H,dv] fp32."""
    return _gla("gla_fwd_f32", q, k, v, log_alpha, Hgrid, Wgrid, direction, out, stream, torch.float32)


def _bwd(fn_name: str, q, k, v, log_alpha, dout, Hgrid, Wgrid, direction, stream, dtype):
    dev = q.device
    for t, n in ((q, "q"), (k, "k"), (v, "v"), (dout, "dout")):
        _need(t, n, dtype, dev)
    _need(log_alpha, "log_alpha", torch.float32, dev)
    if q.dim() != 4 or k.shape != q.shape or log_alpha.shape != q.shape or v.dim() != 4 or v.shape[:3] != q.shape[:3]:
        raise ValueError("expected q, k, log_alpha [B,T,H,dk] and v [B,T,H,dv]")
    if dout.shape != v.shape:
        raise ValueError("dout must be [B,T,H,dv]")
    B, T, H, dk = q.shape
    dv = v.shape[3]
    if T != Hgrid * Wgrid:
        raise ValueError(f"T={T} does not match the grid {Hgrid}x{Wgrid}")
    dq, dk_, dv_ = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    dla = torch.empty_like(log_alpha)
    with torch.cuda.device(dev):
        rc = getattr(_lib, fn_name)(q.data_ptr(), k.data_ptr(), v.data_ptr(), log_alpha.data_ptr(), dout.data_ptr(),
                                    B, H, Hgrid, Wgrid, dk, dv, int(direction), dq.data_ptr(), dk_.data_ptr(),
                                    dv_.data_ptr(), dla.data_ptr(), _stream_handle(dev, stream))
    _check(fn_name, rc)
    return dq, dk_, dv_, dla


def gla_bwd(q, k, v, log_alpha, dout, Hgrid: int, Wgrid: int, direction: int, stream=None):
    """bf16 GLA backward (see include/dig_gla.h, gla_bwd): the gradients of sum(dout * out)
    for out = gla_fwd(q, k, v, log_alpha, ...).  Returns (dq, dk, dv) bf16 and dlog_alpha fp32."""
    return _bwd("gla_bwd", q, k, v, log_alpha, dout, Hgrid, Wgrid, direction, stream, torch.bfloat16)


def gla_bwd_f32(q, k, v, log_alpha, dout, Hgrid: int, Wgrid: int, direction: int, stream=None):
    """fp32 GLA backward (see include/dig_gla.h, gla_bwd_f32).  Returns (dq, dk, dv, dlog_alpha) fp32."""
    return _bwd("gla_bwd_f32", q, k, v, log_alpha, dout, Hgrid, Wgrid, direction, stream, torch.float32)


def _norm(fn_name, q, k, v, Hgrid, Wgrid, direction, eps, out, stream, dtype):
    dev = q.device
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _need(t, n, dtype, dev)
    if q.dim() != 4 or k.shape != q.shape or v.dim() != 4 or v.shape[:3] != q.shape[:3]:
        raise ValueError("expected q, k [B,T,H,dk] and v [B,T,H,dv]")
    B, T, H, dk = q.shape
    dv = v.shape[3]
    if T != Hgrid * Wgrid:
        raise ValueError(f"T={T} does not match the grid {Hgrid}x{Wgrid}")
    if out is None:
        out = torch.empty_like(v)
    else:
        _need(out, "out", dtype, dev)
        if out.shape != v.shape:
            raise ValueError("out must be [B,T,H,dv]")
    with torch.cuda.device(dev):
        rc = getattr(_lib, fn_name)(q.data_ptr(), k.data_ptr(), v.data_ptr(), B, H, Hgrid, Wgrid, dk, dv,
                                    int(direction), float(eps), out.data_ptr(), _stream_handle(dev, stream))
    _check(fn_name, rc)
    return out


def gla_norm_fwd(q, k, v, Hgrid: int, Wgrid: int, direction: int, eps: float = 1e-6, out=None, stream=None):
    """The draft's normalised GLA, bf16 (see include/dig_gla.h, gla_norm_fwd)."""
    return _norm("gla_norm_fwd", q, k, v, Hgrid, Wgrid, direction, eps, out, stream, torch.bfloat16)


def gla_norm_fwd_f32(q, k, v, Hgrid: int, Wgrid: int, direction: int, eps: float = 1e-6, out=None, stream=None):
    """The draft's normalised GLA, fp32 (see include/dig_gla.h, gla_norm_fwd_f32)."""
    return _norm("gla_norm_fwd_f32", q, k, v, Hgrid, Wgrid, direction, eps, out, stream, torch.float32)


def _grid_dtype(x: torch.Tensor) -> int:
    if x.dtype == torch.bfloat16:
        return _BF16
    if x.dtype == torch.float32:
        return _F32
    raise TypeError("grid tensors must be bf16 or fp32")


def srem_reorient(x, direction: int, inverse: int, Hgrid: int, Wgrid: int, out=None, stream=None):
    """Row gather into (inverse=0) or out of (inverse=1) the scan order.  x: [B, T, C] or [B, Hg, Wg, C]."""
    dt = _grid_dtype(x)
    _need(x, "x", x.dtype, x.device)
    B = x.shape[0]
    C = x.shape[-1]
    if x.numel() != B * Hgrid * Wgrid * C:
        raise ValueError("x must hold B x Hgrid x Wgrid x C elements")
    if out is None:
        out = torch.empty_like(x)
    else:
        _need(out, "out", x.dtype, x.device)
        if out.numel() != x.numel():
            raise ValueError("out must match x")
    with torch.cuda.device(x.device):
        rc = _lib.srem_reorient(x.data_ptr(), int(direction), int(inverse), B, Hgrid, Wgrid, C, dt, out.data_ptr(),
                                _stream_handle(x.device, stream))
    _check("srem_reorient", rc)
    return out


def dwconv3x3(x, w, out=None, stream=None):
    """Depthwise 3x3 conv, zero padding.  x: [B, Hg, Wg, C] bf16/fp32 channels-last; w: [C, 3, 3] fp32."""
    dt = _grid_dtype(x)
    _need(x, "x", x.dtype, x.device)
    _need(w, "w", torch.float32, x.device)
    if x.dim() != 4 or tuple(w.shape) != (x.shape[3], 3, 3):
        raise ValueError("expected x [B,Hg,Wg,C] and w [C,3,3]")
    B, Hg, Wg, C = x.shape
    if out is None:
        out = torch.empty_like(x)
    else:
        _need(out, "out", x.dtype, x.device)
        if out.shape != x.shape:
            raise ValueError("out must match x")
    with torch.cuda.device(x.device):
        rc = _lib.dwconv3x3(x.data_ptr(), w.data_ptr(), B, Hg, Wg, C, dt, out.data_ptr(),
                            _stream_handle(x.device, stream))
    _check("dwconv3x3", rc)
    return out


# ---- gated linear recurrence (vector state) -----------------------------------------


# A call of a small shape is bound by the host, so the checks below read each property of a
# tensor once and leave the wording of a refusal to _refuse.
_Tensor = torch.Tensor


def _refuse(t, name: str, dtype: torch.dtype, dev: torch.device, contiguous: bool = True):
    """Raises what is wrong with t; ValueError about its layout if nothing else is."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device != dev or dev.type != "cuda":
        raise ValueError(f"{name} must be on {dev if dev.type == 'cuda' else 'a CUDA device'} (got {t.device})")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype} (got {t.dtype})")
    raise ValueError(f"{name} must be contiguous" if contiguous else f"{name}: unsupported layout")


def _on(t, name: str, dtype: torch.dtype, dev: torch.device, index: int):
    if not (isinstance(t, _Tensor) and t.dtype is dtype and t.get_device() == index >= 0):
        _refuse(t, name, dtype, dev, False)


def _dense(t, name: str, dtype: torch.dtype, dev: torch.device, index: int, shape):
    """Checks a dense tensor of a given shape."""
    if not (isinstance(t, _Tensor) and t.dtype is dtype and t.get_device() == index >= 0 and t.is_contiguous()):
        _refuse(t, name, dtype, dev)
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)} (got {list(t.shape)})")


def _new(t):
    """A dense tensor of t's shape and type."""
    return torch.empty_like(t) if t.is_contiguous() else torch.empty_like(t, memory_format=torch.contiguous_format)


def _row_stride(t: torch.Tensor, name: str, lead: int, inner: int) -> int:
    """Elements between token rows of t, whose first `lead` dimensions are tokens (batches
    behind one another without a gap) and whose other dimensions are dense, `inner` elements."""
    if t.is_contiguous():
        return inner
    shape, stride = t.shape, t.stride()
    dense = 1
    for d in range(len(shape) - 1, lead - 1, -1):
        if shape[d] != 1 and stride[d] != dense:
            raise ValueError(f"{name}: the channels of a token must be contiguous")
        dense *= shape[d]
    step, tokens = None, 1
    for d in range(lead - 1, -1, -1):
        if shape[d] != 1:
            if step is None:
                step = stride[d]
            elif stride[d] != step * tokens:
                raise ValueError(f"{name}: its tokens must be equally spaced in memory")
        tokens *= shape[d]
    return inner if step is None else step


def _ptr(t) -> int | None:
    return None if t is None else t.data_ptr()


# The current device and its current stream without the Stream object that
# torch.cuda.current_stream builds (a microsecond a call).
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _call(fn, dev: torch.device, index: int, stream, *args):
    """fn(*args, stream) with `dev` current; an error status raises."""
    if index == _current_device():
        rc = fn(*args, _raw_stream(index) if stream is None else _stream_handle(dev, stream))
    else:
        with torch.cuda.device(dev):
            rc = fn(*args, _stream_handle(dev, stream))
    if rc != 0:
        raise GlaError(fn.__name__, rc)


def _gated(x, gate, gate_norm, dims: int):
    """Checks x and gate; (device, its index, shape, dtype code, gate_norm for the C call, row strides)."""
    if not isinstance(x, _Tensor):
        raise TypeError("x must be a torch.Tensor")
    dtype, dev, index, shape = x.dtype, x.device, x.get_device(), x.shape
    dt = _grid_dtype(x)
    if index < 0:
        _refuse(x, "x", dtype, dev)
    if gate_norm is None:
        norm, gtype = 0.0, torch.float32
    else:
        norm, gtype = float(gate_norm), dtype
        if not 1e-30 <= norm <= 1e38:  # as fp32, where 0 would mean log_alpha
            raise ValueError("gate_norm must be in [1e-30, 1e38] (None: gate holds log_alpha)")
    _on(gate, "gate", gtype, dev, index)
    if len(shape) != dims or gate.shape != shape:
        raise ValueError(f"expected x and gate of the same {dims}-dimensional shape")
    if x.numel() >= 1 << 31 and max(shape) >= 1 << 31:
        raise ValueError("x: a dimension of 2^31 or more")
    C = shape[-1]
    return dev, index, shape, dt, norm, _row_stride(x, "x", dims - 1, C), _row_stride(gate, "gate", dims - 1, C)


def _grid_sizes(shape, Hgrid, Wgrid):
    if shape[1] != Hgrid * Wgrid:
        raise ValueError(f"T={shape[1]} does not match the grid {Hgrid}x{Wgrid}")
    return (shape[0], Hgrid, Wgrid, shape[2]), shape[0]


def _packed_sizes(shape, cu, dev, index):
    n = cu.numel() - 1 if isinstance(cu, _Tensor) else 0
    _dense(cu, "cu_seqlens", torch.int32, dev, index, (n + 1,))
    if n < 1:
        raise ValueError("cu_seqlens must be [sequences + 1]")
    return (shape[0], n, shape[1]), n


def _glr_fwd(fn, x, gate, where, direction, gate_norm, complement, h0, out, h_last, stream):
    packed = len(where) == 1
    dev, index, shape, dt, norm, xs, gs = _gated(x, gate, gate_norm, 2 if packed else 3)
    sizes, n = _packed_sizes(shape, where[0], dev, index) if packed else _grid_sizes(shape, *where)
    states = (n, shape[-1])
    if h0 is not None:
        _dense(h0, "h0", torch.float32, dev, index, states)
    fill = out is None
    if fill:
        out = _new(x)
    else:
        _dense(out, "out", x.dtype, dev, index, shape)
    if h_last is None:
        h_last = torch.empty(states, dtype=torch.float32, device=dev) if h0 is None else torch.empty_like(h0)
    else:
        _dense(h_last, "h_last", torch.float32, dev, index, states)
    _call(fn, dev, index, stream, x.data_ptr(), gate.data_ptr(), *((where[0].data_ptr(),) if packed else ()), _ptr(h0),
          *sizes, xs, gs, int(direction), norm, int(bool(complement)), dt, *((int(fill),) if packed else ()),
          out.data_ptr(), h_last.data_ptr())
    return out, h_last


def glr_fwd(x, gate, Hgrid: int, Wgrid: int, direction: int, gate_norm: float | None = None, complement: bool = False,
            h0=None, out=None, h_last=None, stream=None):
    """Gated linear recurrence h_p = alpha_p h_{p-1} + s_p x_p over the scan order of a grid (see
    include/dig_gla.h, glr_fwd).  x [B,T,C] bf16 or fp32, possibly a slice of a wider projection;
    gate [B,T,C]: log_alpha in fp32 (gate_norm None), or logits of x's type with log_alpha =
    logsigmoid(gate) / gate_norm.  complement: s = 1 - alpha instead of 1.  h0 [B,C] fp32.
    Returns (out [B,T,C], h_last [B,C] fp32); h_last may be given as h0 to carry a state in place."""
    return _glr_fwd(_lib.glr_fwd, x, gate, (Hgrid, Wgrid), direction, gate_norm, complement, h0, out, h_last, stream)


def glr_fwd_packed(x, gate, cu_seqlens, direction: int = 0, gate_norm: float | None = None, complement: bool = False,
                   h0=None, out=None, h_last=None, stream=None):
    """glr_fwd over packed sequences: x, gate [rows,C], cu_seqlens int32 [n+1] on the device,
    direction 0 or 1, h0 and h_last [n,C].  Rows of no sequence: left as they were in a given
    `out`, zero in a new one."""
    return _glr_fwd(_lib.glr_fwd_packed, x, gate, (cu_seqlens,), direction, gate_norm, complement, h0, out, h_last, stream)


def _glr_bwd(fn, x, gate, h, dout, where, direction, gate_norm, complement, h0, dh_last, outs, stream):
    packed = len(where) == 1
    dev, index, shape, dt, norm, xs, gs = _gated(x, gate, gate_norm, 2 if packed else 3)
    sizes, n = _packed_sizes(shape, where[0], dev, index) if packed else _grid_sizes(shape, *where)
    states = (n, shape[-1])
    _dense(h, "h", x.dtype, dev, index, shape)
    _dense(dout, "dout", x.dtype, dev, index, shape)
    if h0 is not None:
        _dense(h0, "h0", torch.float32, dev, index, states)
    if dh_last is not None:
        _dense(dh_last, "dh_last", torch.float32, dev, index, states)
    dx, dgate, dh0 = outs
    if packed and (dx is None) != (dgate is None):
        raise ValueError("give both dx and dgate, or neither")
    fill = dx is None
    if fill:
        dx = _new(x)
    else:
        _dense(dx, "dx", x.dtype, dev, index, shape)
    if dgate is None:
        dgate = _new(gate)
    else:
        _dense(dgate, "dgate", gate.dtype, dev, index, shape)
    if dh0 is None:
        dh0 = torch.empty(states, dtype=torch.float32, device=dev) if h0 is None else torch.empty_like(h0)
    else:
        _dense(dh0, "dh0", torch.float32, dev, index, states)
    _call(fn, dev, index, stream, x.data_ptr(), gate.data_ptr(), h.data_ptr(), dout.data_ptr(),
          *((where[0].data_ptr(),) if packed else ()), _ptr(h0), _ptr(dh_last), *sizes, xs, gs, int(direction), norm,
          int(bool(complement)), dt, *((int(fill),) if packed else ()), dx.data_ptr(), dgate.data_ptr(), dh0.data_ptr())
    return dx, dgate, dh0


def glr_bwd(x, gate, h, dout, Hgrid: int, Wgrid: int, direction: int, gate_norm: float | None = None,
            complement: bool = False, h0=None, dh_last=None, dx=None, dgate=None, dh0=None, stream=None):
    """The gradients of sum(dout * out) + sum(dh_last * h_last) for (out, h_last) = glr_fwd(x, gate,
    ...), with h = that out (see include/dig_gla.h, glr_bwd).  Returns (dx of x's type, dgate of
    gate's type, dh0 fp32 [B,C])."""
    return _glr_bwd(_lib.glr_bwd, x, gate, h, dout, (Hgrid, Wgrid), direction, gate_norm, complement, h0, dh_last,
                    (dx, dgate, dh0), stream)


def glr_bwd_packed(x, gate, h, dout, cu_seqlens, direction: int = 0, gate_norm: float | None = None,
                   complement: bool = False, h0=None, dh_last=None, dx=None, dgate=None, dh0=None, stream=None):
    """glr_bwd over packed sequences.  Rows of no sequence: left as they were in given dx and
    dgate, zero in new ones."""
    return _glr_bwd(_lib.glr_bwd_packed, x, gate, h, dout, (cu_seqlens,), direction, gate_norm, complement, h0, dh_last,
                    (dx, dgate, dh0), stream)


def glr_step(x, gate, state, slots=None, gate_norm: float | None = None, complement: bool = False, state_out=None,
             out=None, stream=None):
    """One token of the recurrence for every row (see include/dig_gla.h, glr_step).  x, gate [N,C];
    state [nslots,C] fp32; slots int32 [N] (None: row i uses state i; negative: a padded row).
    Updates `state` in place, or writes the new states to `state_out`.  Returns (out [N,C], the
    updated pool); padded rows are left as they were in a given `out`, zero in a new one."""
    dev, index, shape, dt, norm, xs, gs = _gated(x, gate, gate_norm, 2)
    N, C = shape
    nslots = state.shape[0] if isinstance(state, _Tensor) and state.dim() else 0
    pool = (nslots, C)
    _dense(state, "state", torch.float32, dev, index, pool)
    if slots is not None:
        _dense(slots, "slots", torch.int32, dev, index, (N,))
    fill = out is None
    if fill:
        out = _new(x)
    else:
        _dense(out, "out", x.dtype, dev, index, shape)
    if state_out is None:
        state_out = state
    else:
        _dense(state_out, "state_out", torch.float32, dev, index, pool)
    _call(_lib.glr_step, dev, index, stream, x.data_ptr(), gate.data_ptr(), state.data_ptr(), _ptr(slots), N, nslots, C,
          xs, gs, norm, int(bool(complement)), dt, int(fill), state_out.data_ptr(), out.data_ptr())
    return out, state_out


# ---- rotary positions, query/key norm ------------------------------------------------


def rope_frequencies(rot: int, base: float = 10000.0, scaling: str | None = None, factor: float = 1.0,
                     original_length: int = 0, beta_fast: float = 32.0, beta_slow: float = 1.0, device=None):
    """The inv_freq table [rot/2] (fp32) and the scale of rope and qk_norm_rope.

    Unscaled, inv_freq[i] = base^(-2i/rot).  For contexts `factor` times longer than the
    `original_length` the weights were trained on:
      "linear"  positions shrink: inv_freq / factor
      "base"    the base grows so that the slowest pair alone slows down by factor:
                base * factor^(rot / (rot - 2))
      "ramp"    pairs that turn more than beta_fast times over original_length keep their
                frequency, those that turn less than beta_slow times are divided by
                factor, in between the two are blended linearly in i; scale = 0.1 ln(factor) + 1
                (the by-parts interpolation of YaRN, Peng et al. 2023)
    """
    if rot <= 0 or rot % 2:
        raise ValueError("rot must be positive and even")
    if not base > 0 or not factor >= 1:
        raise ValueError("base must be positive and factor at least 1")
    if scaling not in (None, "linear", "base", "ramp"):
        raise ValueError('scaling must be None, "linear", "base" or "ramp"')
    i = torch.arange(rot // 2, dtype=torch.float64)
    scale = 1.0
    if scaling == "base":
        if rot < 4:
            raise ValueError('scaling "base" needs rot >= 4')
        base = base * factor ** (rot / (rot - 2))
    inv = torch.pow(torch.tensor(base, dtype=torch.float64), -2.0 * i / rot)
    if scaling == "linear":
        inv = inv / factor
    elif scaling == "ramp":
        if original_length <= 0 or not beta_fast > beta_slow > 0 or not base > 1:
            raise ValueError('scaling "ramp" needs original_length, base > 1 and beta_fast > beta_slow > 0')

        def pair_of(turns):  # the (fractional) pair that turns so often over original_length
            return rot * math.log(original_length / (turns * 2 * math.pi)) / (2 * math.log(base))

        # Either end may lie outside the table: cut to it, the slope inside would be another.
        low, high = math.floor(pair_of(beta_fast)), math.ceil(pair_of(beta_slow))
        slow = torch.clamp((i - low) / max(high - low, 1), 0, 1)
        inv = inv * (1 - slow) + inv / factor * slow
        scale = 0.1 * math.log(factor) + 1.0
    return inv.to(torch.float32).to("cpu" if device is None else device), scale


def _heads(t, name: str, dtype, dev, index: int, like):
    """Checks a tensor of heads [*rows, H, D] whose rows and D are those of the shape `like`;
    (H, its row stride)."""
    if not (isinstance(t, _Tensor) and t.dtype is dtype and t.get_device() == index):
        _refuse(t, name, dtype, dev, False)
    shape = t.shape
    n = len(like)
    if len(shape) != n or shape[0] != like[0] or shape[-1] != like[-1] or (n == 4 and shape[1] != like[1]):
        raise ValueError(f"{name}: expected [rows,H,D] or [B,T,H,D] with the rows and D of the queries")
    H, D = shape[-2], shape[-1]
    if t.is_contiguous():
        return H, H * D
    if n == 3:
        stride = t.stride()
        if stride[2] == 1 and stride[1] == D and shape[0] != 1:
            return H, stride[0]
    return H, _row_stride(t, name, n - 2, H * D)


def _head_out(t, name: str, like, dtype, dev, index: int, H: int):
    """A caller's output of `like`'s shape, or a new dense one; with its row stride."""
    if t is None:
        return _new(like), H * like.shape[-1]
    h, stride = _heads(t, name, dtype, dev, index, like.shape)
    if h != H:
        raise ValueError(f"{name} must be {list(like.shape)} (got {list(t.shape)})")
    return t, stride


def _queries(q):
    """(device, its index, dtype, dtype code, shape, rows) of the queries."""
    if not isinstance(q, _Tensor):
        raise TypeError("q must be a torch.Tensor")
    dt, shape, dev, index = _grid_dtype(q), q.shape, q.device, q.get_device()
    if len(shape) not in (3, 4):
        raise ValueError("q: expected [rows,H,D] or [B,T,H,D]")
    if index < 0:
        _refuse(q, "q", q.dtype, dev)
    return dev, index, q.dtype, dt, shape, shape[0] if len(shape) == 3 else shape[0] * shape[1]


def _angle_args(positions, inv_freq, dev, index, shape, rows):
    """C arguments of the positions and the table, and rot."""
    at, wide = None, 0
    if positions is not None:
        if not isinstance(positions, _Tensor) or positions.dtype not in (torch.int32, torch.int64):
            raise TypeError("positions must be an int32 or int64 tensor")
        wide = int(positions.dtype is torch.int64)
        if positions.get_device() != index or not positions.is_contiguous():
            _refuse(positions, "positions", positions.dtype, dev)
        if positions.shape != shape[:-2]:
            raise ValueError("positions must be one for each row of q")
        at = positions.data_ptr()
    rot, table = 0, None
    if inv_freq is not None:
        if not (isinstance(inv_freq, _Tensor) and inv_freq.dtype is torch.float32 and inv_freq.get_device() == index
                and inv_freq.is_contiguous()):
            _refuse(inv_freq, "inv_freq", torch.float32, dev)
        if inv_freq.dim() != 1:
            raise ValueError("inv_freq must be [rot/2]")
        rot, table = 2 * inv_freq.numel(), inv_freq.data_ptr()
    return (at, wide, shape[-3], table, rows), rot


def _rope_call(fn, q, k, weights, positions, inv_freq, middle, q_out, k_out, stream):
    dev, index, dtype, dt, shape, rows = _queries(q)
    D = shape[-1]
    angles, rot = _angle_args(positions, inv_freq, dev, index, shape, rows)
    w = _weights(k, *weights, dev, index, D) if weights else ()
    H, qs = _heads(q, "q", dtype, dev, index, shape)
    q_out, qos = _head_out(q_out, "q_out", q, dtype, dev, index, H)
    Hk, ks, kos, pk, pko = 0, D, D, None, None
    if k is not None:
        Hk, ks = _heads(k, "k", dtype, dev, index, shape)
        k_out, kos = _head_out(k_out, "k_out", k, dtype, dev, index, Hk)
        pk, pko = k.data_ptr(), k_out.data_ptr()
    elif k_out is not None:
        raise ValueError("k_out without k")
    _call(fn, dev, index, stream, q.data_ptr(), pk, *w, *angles, H, Hk, D, rot, qs, ks, *middle, dt, q_out.data_ptr(), qos,
          pko, kos)
    return q_out, k_out


def rope(q, k, positions, inv_freq, interleaved: bool = False, scale: float = 1.0, inverse: bool = False, q_out=None,
         k_out=None, stream=None):
    """Rotary positions of query and key heads (see include/dig_gla.h, rope).  q [rows,Hq,D] or
    [B,T,Hq,D], k likewise with Hk heads or None, bf16 or fp32, possibly slices of one fused
    projection; positions int32/int64, one a row (None: 0..T-1 in every batch); inv_freq
    fp32 [rot/2] (rope_frequencies).  inverse: turns back, the gradient.  q_out, k_out may be q
    and k.  Returns (q_out, k_out)."""
    return _rope_call(_lib.rope, q, k, (), positions, inv_freq, (int(bool(interleaved)), int(bool(inverse)), float(scale)),
                      q_out, k_out, stream)


def _weights(k, q_weight, k_weight, dev, index, D):
    _dense(q_weight, "q_weight", torch.float32, dev, index, (D,))
    if k is not None:
        _dense(k_weight, "k_weight", torch.float32, dev, index, (D,))
        return q_weight.data_ptr(), k_weight.data_ptr()
    if k_weight is not None:
        raise ValueError("k_weight without its heads")
    return q_weight.data_ptr(), None


def qk_norm_rope(q, k, q_weight, k_weight, positions, inv_freq, eps: float = 1e-6, interleaved: bool = False,
                 scale: float = 1.0, q_out=None, k_out=None, stream=None):
    """RMS norm of every query and key head, then rope, in one pass (see include/dig_gla.h,
    qk_norm_rope).  q_weight, k_weight fp32 [D]; inv_freq None: the norm alone.  The rest as rope.
    Returns (q_out, k_out)."""
    return _rope_call(_lib.qk_norm_rope, q, k, (q_weight, k_weight), positions, inv_freq,
                      (int(bool(interleaved)), float(eps), float(scale)), q_out, k_out, stream)


def qk_norm_rope_bwd(dq_out, dk_out, q, k, q_weight, k_weight, positions, inv_freq, eps: float = 1e-6,
                     interleaved: bool = False, scale: float = 1.0, dq=None, dk=None, stream=None):
    """The gradients of qk_norm_rope (see include/dig_gla.h, qk_norm_rope_bwd) from its inputs and
    those of its outputs.  dq and dk may be dq_out and dk_out.  Returns (dq, dk, dq_weight fp32,
    dk_weight fp32)."""
    dev, index, dtype, dt, shape, rows = _queries(q)
    D = shape[-1]
    angles, rot = _angle_args(positions, inv_freq, dev, index, shape, rows)
    w = _weights(k, q_weight, k_weight, dev, index, D)
    H, qs = _heads(q, "q", dtype, dev, index, shape)
    h, dqs = _heads(dq_out, "dq_out", dtype, dev, index, shape)
    if h != H:
        raise ValueError("dq_out must have q's shape")
    dq, dqo = _head_out(dq, "dq", q, dtype, dev, index, H)
    dwq = torch.empty_like(q_weight)
    Hk, ks, dks, dko, dwk = 0, D, D, D, None
    if k is not None:
        Hk, ks = _heads(k, "k", dtype, dev, index, shape)
        h, dks = _heads(dk_out, "dk_out", dtype, dev, index, shape)
        if h != Hk:
            raise ValueError("dk_out must have k's shape")
        dk, dko = _head_out(dk, "dk", k, dtype, dev, index, Hk)
        dwk = torch.empty_like(k_weight)
    elif dk_out is not None or dk is not None:
        raise ValueError("dk_out or dk without k")
    _call(_lib.qk_norm_rope_bwd, dev, index, stream, dq_out.data_ptr(), _ptr(dk_out), q.data_ptr(), _ptr(k), *w, *angles, H,
          Hk, D, rot, dqs, dks, qs, ks, int(bool(interleaved)), float(eps), float(scale), dt, dq.data_ptr(), dqo, _ptr(dk),
          dko, dwq.data_ptr(), _ptr(dwk))
    return dq, dk, dwq, dwk


def skip_items_for_test(n: int) -> None:
    """Test hook: the next gla_fwd call leaves out its first n work items, so the
    look-back waits that need them run out (device status GLA_ERR_TIMEOUT afterwards,
    output unspecified).  n <= 0 clears it."""
    _lib.dig_gla_test_skip_items(int(n))


def device_status(stream=None, device=None) -> int:
    """Synchronise the stream, then return and clear the device status word (0 = GLA_OK)."""
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    with torch.cuda.device(dev):
        return int(_lib.dig_gla_device_status(_stream_handle(dev, stream)))
