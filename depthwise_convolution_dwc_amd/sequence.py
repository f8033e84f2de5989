"""Operators of the sequence layer around a depthwise convolution: layer
norm, dropout from a counter-based generator and the gated delta rule, on
torch tensors.  Argument marshalling only, like the package's other calls;
the formulas stand in include/dwc.h.

Every call runs on the current stream of the tensors' device, or on
``stream``; outputs and workspaces that a call allocates are then recorded
on that stream, so that the allocator does not hand them out too early.
"""

from __future__ import annotations

import ctypes
import math
from typing import Optional, Tuple

import torch

from . import _DTYPE_CODE, _raise, lib

DELTA_FWD, DELTA_BWD = 0, 1
_TYPES = (torch.float32, torch.bfloat16, torch.float16)
_I3 = ctypes.c_int64 * 3


class NormProblem(ctypes.Structure):
    """Mirror of ``dwc_norm_problem`` in include/dwc.h."""

    _fields_ = [("rows", ctypes.c_int64), ("c", ctypes.c_int64), ("x_stride", ctypes.c_int64),
                ("dy_stride", ctypes.c_int64), ("x_dtype", ctypes.c_int32),
                ("y_dtype", ctypes.c_int32), ("w_dtype", ctypes.c_int32), ("eps", ctypes.c_float)]


class DropoutProblem(ctypes.Structure):
    """Mirror of ``dwc_dropout_problem``."""

    _fields_ = [("n", ctypes.c_int64), ("p", ctypes.c_double), ("seed", ctypes.c_uint64),
                ("offset", ctypes.c_uint64), ("dtype", ctypes.c_int32),
                ("reserved", ctypes.c_int32)]


class DeltaProblem(ctypes.Structure):
    """Mirror of ``dwc_delta_problem``."""

    _fields_ = [("b", ctypes.c_int64), ("l", ctypes.c_int64), ("q_stride", _I3),
                ("k_stride", _I3), ("v_stride", _I3), ("g_stride", _I3), ("beta_stride", _I3),
                ("do_stride", _I3), ("hk", ctypes.c_int32), ("hv", ctypes.c_int32),
                ("dk", ctypes.c_int32), ("dv", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("scale", ctypes.c_float)]


def bind(l: ctypes.CDLL) -> None:
    """Argument types of the sequence-layer entry points."""
    vp, sz = ctypes.c_void_p, ctypes.c_size_t
    n, d, r = (ctypes.POINTER(t) for t in (NormProblem, DropoutProblem, DeltaProblem))
    l.dwc_layer_norm.argtypes = [n] + [vp] * 7
    l.dwc_layer_norm_bwd_workspace_size.argtypes = [n, ctypes.POINTER(sz)]
    l.dwc_layer_norm_bwd.argtypes = [n] + [vp] * 9 + [sz, vp]
    l.dwc_dropout.argtypes = [d] + [vp] * 4
    l.dwc_delta_step.argtypes = [r] + [vp] * 10
    l.dwc_delta_workspace_size.argtypes = [r, ctypes.c_int, ctypes.POINTER(sz)]
    l.dwc_delta_fwd.argtypes = [r] + [vp] * 10 + [sz, vp]
    l.dwc_delta_bwd.argtypes = [r] + [vp] * 16 + [sz, vp]


class _On:
    """The device of ``t`` made current, and the stream to launch on."""

    def __init__(self, t: torch.Tensor, stream):
        self._guard = torch.cuda.device(t.device) \
            if t.device.index != torch.cuda.current_device() else None
        self._stream = stream
        self._given = stream is not None

    def __enter__(self):
        if self._guard is not None:
            self._guard.__enter__()
        s = self._stream
        if s is None:
            return torch.cuda.current_stream().cuda_stream
        return s.cuda_stream if hasattr(s, "cuda_stream") else int(s)

    def __exit__(self, *exc):
        if self._guard is not None:
            self._guard.__exit__(*exc)

    def made(self, *ts):
        """Marks tensors allocated here as used on the stream given."""
        if self._given:
            s = self._stream
            if not hasattr(s, "cuda_stream"):
                s = torch.cuda.ExternalStream(int(s))
            for t in ts:
                if t is not None:
                    t.record_stream(s)


def _device_tensor(t, name, dtypes=None, device=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if device is not None and t.device != device:
        raise ValueError(f"{name} must be on {device}, got {t.device}")
    if dtypes is not None and t.dtype not in dtypes:
        raise TypeError(f"{name} must be one of {dtypes}, got {t.dtype}")


def _dense(t, name, shape):
    if tuple(t.shape) != tuple(shape) or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous of shape {tuple(shape)}, "
                         f"got {tuple(t.shape)}")


def _ptr(t):
    return t.data_ptr() if t is not None else None


def _row_stride(t, name):
    """Elements between the rows of (..., c) seen as rows x c; raises where
    the leading axes do not form one stride or the last is not dense."""
    c = t.shape[-1]
    if t.numel() == 0:
        return c
    if c > 1 and t.stride(-1) != 1:
        raise ValueError(f"{name}'s last axis must be dense")
    stride, span = None, None
    for n, st in zip(reversed(t.shape[:-1]), reversed(t.stride()[:-1])):
        if n == 1:
            continue
        if stride is None:
            stride = st
        elif st != span:
            raise ValueError(f"{name}'s leading axes must form one row stride")
        span = st * n
    stride = c if stride is None else stride
    if stride < c:
        raise ValueError(f"{name}'s rows overlap")
    return stride


def _weights(w, b, c, device):
    for t, name in ((w, "w"), (b, "b")):
        if t is not None:
            _device_tensor(t, name, _TYPES, device)
            _dense(t, name, (c,))
    if w is not None and b is not None and w.dtype != b.dtype:
        raise TypeError("w and b must have one dtype")
    t = w if w is not None else b
    return _DTYPE_CODE[t.dtype] if t is not None else 0


def layer_norm(x: torch.Tensor, w: Optional[torch.Tensor] = None,
               b: Optional[torch.Tensor] = None, eps: float = 1e-5,
               out_dtype: Optional[torch.dtype] = None, out: Optional[torch.Tensor] = None,
               stream=None) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """Layer norm over the last axis: (y, mean, rstd), y of ``out_dtype``
    (x's by default), mean and 1 / sqrt(var + eps) fp32, one a row."""
    _device_tensor(x, "x", _TYPES)
    if x.dim() < 1 or x.shape[-1] < 1:
        raise ValueError("x needs a last axis of at least one element")
    c, lead = x.shape[-1], x.shape[:-1]
    rows = x.numel() // c
    wt = _weights(w, b, c, x.device)
    if out is not None:
        _device_tensor(out, "out", _TYPES if out_dtype is None else (out_dtype,), x.device)
        _dense(out, "out", x.shape)
        out_dtype = out.dtype
    out_dtype = out_dtype or x.dtype
    if out_dtype not in _TYPES:
        raise TypeError(f"out_dtype must be one of {_TYPES}, got {out_dtype}")
    p = NormProblem(rows, c, _row_stride(x, "x"), c, _DTYPE_CODE[x.dtype],
                    _DTYPE_CODE[out_dtype], wt, eps)
    on = _On(x, stream)
    with on as s:
        made = out is None
        if made:
            out = torch.empty(x.shape, dtype=out_dtype, device=x.device)
        mean = torch.empty(lead, dtype=torch.float32, device=x.device)
        rstd = torch.empty(lead, dtype=torch.float32, device=x.device)
        on.made(out if made else None, mean, rstd)
        _raise(lib().dwc_layer_norm(ctypes.byref(p), _ptr(x), _ptr(w), _ptr(b), _ptr(out),
                                    _ptr(mean), _ptr(rstd), s))
    return out, mean, rstd


def layer_norm_bwd(dy: torch.Tensor, x: torch.Tensor, mean: torch.Tensor, rstd: torch.Tensor,
                   w: Optional[torch.Tensor] = None, stream=None
                   ) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """Gradients of ``layer_norm``: (dx of x's dtype, dw, db fp32)."""
    _device_tensor(x, "x", _TYPES)
    _device_tensor(dy, "dy", _TYPES, x.device)
    if dy.shape != x.shape:
        raise ValueError("dy and x disagree in shape")
    if x.dim() < 1 or x.shape[-1] < 1:
        raise ValueError("x needs a last axis of at least one element")
    c, lead = x.shape[-1], x.shape[:-1]
    for t, name in ((mean, "mean"), (rstd, "rstd")):
        _device_tensor(t, name, (torch.float32,), x.device)
        _dense(t, name, lead)
    wt = _weights(w, None, c, x.device)
    p = NormProblem(x.numel() // c, c, _row_stride(x, "x"), _row_stride(dy, "dy"),
                    _DTYPE_CODE[x.dtype], _DTYPE_CODE[dy.dtype], wt, 0.0)
    on = _On(x, stream)
    with on as s:
        need = ctypes.c_size_t()
        _raise(lib().dwc_layer_norm_bwd_workspace_size(ctypes.byref(p), ctypes.byref(need)))
        ws = torch.empty(need.value, dtype=torch.uint8, device=x.device)
        dx = torch.empty(x.shape, dtype=x.dtype, device=x.device)
        dw = torch.empty(c, dtype=torch.float32, device=x.device)
        db = torch.empty(c, dtype=torch.float32, device=x.device)
        on.made(ws, dx, dw, db)
        _raise(lib().dwc_layer_norm_bwd(ctypes.byref(p), _ptr(dy), _ptr(x), _ptr(mean),
                                        _ptr(rstd), _ptr(w), _ptr(dx), _ptr(dw), _ptr(db),
                                        _ptr(ws), need.value, s))
    return dx, dw, db


def dropout(x: torch.Tensor, p: float, seed: int, offset: int = 0,
            residual: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
            stream=None) -> torch.Tensor:
    """residual + (kept ? x / (1 - p) : 0), the mask a function of (seed,
    offset, element index).  The gradient of x is this call on dy with the
    same p, seed and offset; elements of later calls that must not share a
    mask take an offset at least (numel + 3) // 4 further."""
    _device_tensor(x, "x", _TYPES)
    if not x.is_contiguous():
        raise ValueError("x must be contiguous")
    if residual is not None:
        _device_tensor(residual, "residual", (x.dtype,), x.device)
        _dense(residual, "residual", x.shape)
    if not 0 <= int(seed) < 1 << 64 or not 0 <= int(offset) < 1 << 64:
        raise ValueError("seed and offset must be in 0 .. 2^64 - 1")
    if out is not None:
        _device_tensor(out, "out", (x.dtype,), x.device)
        _dense(out, "out", x.shape)
    d = DropoutProblem(x.numel(), p, int(seed), int(offset), _DTYPE_CODE[x.dtype], 0)
    on = _On(x, stream)
    with on as s:
        if out is None:
            out = torch.empty(x.shape, dtype=x.dtype, device=x.device)
            on.made(out)
        _raise(lib().dwc_dropout(ctypes.byref(d), _ptr(x), _ptr(residual), _ptr(out), s))
    return out


def _strides(t, name, heads, last):
    """(batch, token, head) strides of a b x l x h (x d) tensor."""
    if last and t.shape[-1] > 1 and t.numel() and t.stride(-1) != 1:
        raise ValueError(f"{name}'s last axis must be dense")
    return _I3(*t.stride()[:3])


def _delta(q, k, v, g, beta, s0, lengths, scale, dout=None):
    _device_tensor(q, "q", _TYPES)
    dev, dt = q.device, (q.dtype,)
    _device_tensor(k, "k", dt, dev)
    _device_tensor(v, "v", dt, dev)
    _device_tensor(g, "g", (torch.float32,), dev)
    _device_tensor(beta, "beta", (torch.float32,), dev)
    if q.dim() != 4 or v.dim() != 4:
        raise ValueError("q, k and v must be b x l x heads x head size")
    b, n, hk, dk = q.shape
    hv, dv = v.shape[2:]
    if k.shape != q.shape or v.shape[:2] != q.shape[:2]:
        raise ValueError("q, k and v disagree in shape")
    if g.shape != (b, n, hv) or beta.shape != (b, n, hv):
        raise ValueError(f"g and beta must be {(b, n, hv)}")
    if s0 is not None:
        _device_tensor(s0, "s0", (torch.float32,), dev)
        _dense(s0, "s0", (b, hv, dk, dv))
    if lengths is not None:
        _device_tensor(lengths, "lengths", (torch.int32,), dev)
        _dense(lengths, "lengths", (b,))
    if dout is not None:
        _device_tensor(dout, "dout", dt, dev)
        if dout.shape != v.shape:
            raise ValueError("dout and v disagree in shape")
    if scale is None:
        scale = 1.0 / math.sqrt(dk) if dk else 1.0
    return DeltaProblem(b, n, _strides(q, "q", hk, True), _strides(k, "k", hk, True),
                        _strides(v, "v", hv, True), _strides(g, "g", hv, False),
                        _strides(beta, "beta", hv, False),
                        _strides(dout, "dout", hv, True) if dout is not None else _I3(0, 0, 0),
                        hk, hv, dk, dv, _DTYPE_CODE[q.dtype], scale)


def _workspace(p, op, device):
    need = ctypes.c_size_t()
    _raise(lib().dwc_delta_workspace_size(ctypes.byref(p), op, ctypes.byref(need)))
    return torch.empty(need.value, dtype=torch.uint8, device=device), need.value


def delta_rule_step(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, g: torch.Tensor,
                    beta: torch.Tensor, s0: Optional[torch.Tensor] = None,
                    lengths: Optional[torch.Tensor] = None, scale: Optional[float] = None,
                    out_state: Optional[torch.Tensor] = None, stream=None
                    ) -> Tuple[torch.Tensor, torch.Tensor]:
    """The gated delta rule token by token: (o, s1).  The form for one or a
    few new tokens of each sequence; shapes as ``delta_rule``.  out_state
    may be s0: the state is then updated in place."""
    p = _delta(q, k, v, g, beta, s0, lengths, scale)
    shape = (p.b, p.hv, p.dk, p.dv)
    if out_state is not None:
        _device_tensor(out_state, "out_state", (torch.float32,), q.device)
        _dense(out_state, "out_state", shape)
    on = _On(q, stream)
    with on as s:
        o = torch.empty(v.shape, dtype=v.dtype, device=q.device)
        on.made(o)
        if out_state is None:
            out_state = torch.empty(shape, dtype=torch.float32, device=q.device)
            on.made(out_state)
        _raise(lib().dwc_delta_step(ctypes.byref(p), _ptr(q), _ptr(k), _ptr(v), _ptr(g),
                                    _ptr(beta), _ptr(s0), _ptr(lengths), _ptr(o),
                                    _ptr(out_state), s))
    return o, out_state


def delta_rule(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, g: torch.Tensor,
               beta: torch.Tensor, s0: Optional[torch.Tensor] = None,
               lengths: Optional[torch.Tensor] = None, scale: Optional[float] = None,
               stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """The gated delta rule over whole sequences: (o, s1).

    q, k: b x l x hk x dk; v: b x l x hv x dv (views with a dense last axis,
    such as channel ranges of one tensor, are read in place); g, beta:
    b x l x hv fp32; s0: b x hv x dk x dv fp32 or None; lengths: b int32 or
    None.  o: b x l x hv x dv of v's dtype; s1: the states after the last
    token.  scale defaults to 1 / sqrt(dk)."""
    p = _delta(q, k, v, g, beta, s0, lengths, scale)
    on = _On(q, stream)
    with on as s:
        ws, need = _workspace(p, DELTA_FWD, q.device)
        o = torch.empty(v.shape, dtype=v.dtype, device=q.device)
        s1 = torch.empty((p.b, p.hv, p.dk, p.dv), dtype=torch.float32, device=q.device)
        on.made(ws, o, s1)
        _raise(lib().dwc_delta_fwd(ctypes.byref(p), _ptr(q), _ptr(k), _ptr(v), _ptr(g),
                                   _ptr(beta), _ptr(s0), _ptr(lengths), _ptr(o), _ptr(s1),
                                   _ptr(ws), need, s))
    return o, s1


def delta_rule_bwd(dout: torch.Tensor, ds1: Optional[torch.Tensor], q: torch.Tensor,
                   k: torch.Tensor, v: torch.Tensor, g: torch.Tensor, beta: torch.Tensor,
                   s0: Optional[torch.Tensor] = None, lengths: Optional[torch.Tensor] = None,
                   scale: Optional[float] = None, stream=None):
    """Gradients of ``delta_rule`` from those of o and s1 (None: zero):
    (dq, dk, dv, dg, dbeta, ds0), ds0 None where s0 is."""
    p = _delta(q, k, v, g, beta, s0, lengths, scale, dout)
    if ds1 is not None:
        _device_tensor(ds1, "ds1", (torch.float32,), q.device)
        _dense(ds1, "ds1", (p.b, p.hv, p.dk, p.dv))
    on = _On(q, stream)
    with on as s:
        ws, need = _workspace(p, DELTA_BWD, q.device)
        dq = torch.empty(q.shape, dtype=q.dtype, device=q.device)
        dk = torch.empty(k.shape, dtype=k.dtype, device=q.device)
        dv = torch.empty(v.shape, dtype=v.dtype, device=q.device)
        dg = torch.empty(g.shape, dtype=torch.float32, device=q.device)
        dbeta = torch.empty(g.shape, dtype=torch.float32, device=q.device)
        ds0 = torch.empty_like(s0) if s0 is not None else None
        on.made(ws, dq, dk, dv, dg, dbeta, ds0)
        _raise(lib().dwc_delta_bwd(ctypes.byref(p), _ptr(dout), _ptr(ds1), _ptr(q), _ptr(k),
                                   _ptr(v), _ptr(g), _ptr(beta), _ptr(s0), _ptr(lengths),
                                   _ptr(dq), _ptr(dk), _ptr(dv), _ptr(dg), _ptr(dbeta),
                                   _ptr(ds0), _ptr(ws), need, s))
    return dq, dk, dv, dg, dbeta, ds0


__all__ = ["layer_norm", "layer_norm_bwd", "dropout", "delta_rule", "delta_rule_step",
           "delta_rule_bwd", "NormProblem", "DropoutProblem", "DeltaProblem", "DELTA_FWD",
           "DELTA_BWD"]
