"""Operators of a selective state space layer on torch tensors: the short
causal convolution over tokens, the selective scan, and the norms behind one
block and before the next fused with gate, scale and residual sum.  Argument
marshalling only; the formulas stand in include/dwc.h.

Streams and memory are handled as in ``sequence``: every call runs on the
current stream of the tensors' device, or on ``stream``.
"""

from __future__ import annotations

import ctypes
import struct
from typing import Optional, Tuple

import torch

from . import ACT, _DTYPE_CODE, _raise, lib
from .sequence import (_DENSE, _F32, _I3, _I32, _TYPES, _dense, _device_tensor, _on, _ptr, _raw,
                       _returned, _row_stride, _strides, _written)

SCAN_FWD, SCAN_BWD = 0, 1
# DWC_GATE_*: what is made of the gate of residual_norm
GATE = {"none": 0, "silu": 1, "sigmoid": 2}
_I2 = ctypes.c_int64 * 2


class CausalConvProblem(ctypes.Structure):
    """Mirror of ``dwc_causal_conv_problem`` in include/dwc.h."""

    _fields_ = [("b", ctypes.c_int64), ("l", ctypes.c_int64), ("d", ctypes.c_int64),
                ("x_stride", _I2), ("dy_stride", _I2), ("taps", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("w_dtype", ctypes.c_int32), ("act", ctypes.c_int32)]


class ScanProblem(ctypes.Structure):
    """Mirror of ``dwc_scan_problem``."""

    _fields_ = [("b", ctypes.c_int64), ("l", ctypes.c_int64), ("u_stride", _I2),
                ("delta_stride", _I2), ("z_stride", _I2), ("dy_stride", _I2), ("b_stride", _I3),
                ("c_stride", _I3), ("d", ctypes.c_int32), ("n", ctypes.c_int32),
                ("g", ctypes.c_int32), ("dtype", ctypes.c_int32), ("softplus", ctypes.c_int32),
                ("reserved", ctypes.c_int32)]


class ResNormProblem(ctypes.Structure):
    """Mirror of ``dwc_resnorm_problem``."""

    _fields_ = [("rows", ctypes.c_int64), ("c", ctypes.c_int64), ("x_stride", ctypes.c_int64),
                ("y_stride", ctypes.c_int64), ("gate_stride", ctypes.c_int64),
                ("dr_stride", ctypes.c_int64), ("dh_stride", ctypes.c_int64),
                ("x_dtype", ctypes.c_int32), ("y_dtype", ctypes.c_int32),
                ("w_dtype", ctypes.c_int32), ("act", ctypes.c_int32), ("post", ctypes.c_int32),
                ("pre", ctypes.c_int32), ("eps", ctypes.c_float), ("reserved", ctypes.c_int32)]


# The structures' bytes, packed in one step.
_CONV = struct.Struct("7q4i").pack
_SCAN = struct.Struct("16q6i").pack
_RESNORM = struct.Struct("7q6ifi").pack


def bind(l: ctypes.CDLL) -> None:
    """Argument types of the entry points; a problem may be passed by
    reference or as the structure's bytes."""
    vp, sz = ctypes.c_void_p, ctypes.c_size_t
    l.dwc_causal_conv.argtypes = [vp] * 9
    l.dwc_causal_conv_step.argtypes = [vp] * 9
    l.dwc_causal_conv_bwd_workspace_size.argtypes = [vp, ctypes.POINTER(sz)]
    l.dwc_causal_conv_bwd.argtypes = [vp] * 13 + [sz, vp]
    l.dwc_scan_step.argtypes = [vp] * 14
    l.dwc_scan_workspace_size.argtypes = [vp, ctypes.c_int, ctypes.POINTER(sz)]
    l.dwc_scan_fwd.argtypes = [vp] * 14 + [sz, vp]
    l.dwc_scan_bwd.argtypes = [vp] * 23 + [sz, vp]
    l.dwc_residual_norm.argtypes = [vp] * 12
    l.dwc_residual_norm_bwd_workspace_size.argtypes = [vp, ctypes.POINTER(sz)]
    l.dwc_residual_norm_bwd.argtypes = [vp] * 18 + [sz, vp]


def _token_strides(t, name):
    """(batch, token) strides of a b x l x d tensor."""
    s = t.stride()
    if s[2] != 1 and t.shape[2] > 1 and t.numel():
        raise ValueError(f"{name}'s last axis must be dense")
    return s[:2]


def _token_operand(t, name, dtypes, index, shape):
    """Its strides, checked against the first operand."""
    _device_tensor(t, name, dtypes, index)
    if t.shape != shape:
        raise ValueError(f"{name} and u disagree in shape")
    return _token_strides(t, name)


def _lengths(lengths, b, index):
    if lengths is not None:
        _device_tensor(lengths, "lengths", _I32, index)
        _dense(lengths, "lengths", (b,))


def _workspace(like, size, *args):
    need = ctypes.c_size_t()
    _raise(size(*args, ctypes.byref(need)))
    return like.new_empty(need.value, dtype=torch.uint8), need.value


# ---------------------------------------------------------- causal convolution ----

def _conv(x, w, bias, s0, lengths, act, dy=None):
    """(the problem's bytes, device index, shape of the states)"""
    index = _device_tensor(x, "x", _TYPES)
    if x.dim() != 3:
        raise ValueError("x must be b x l x d")
    b, n, d = x.shape
    _device_tensor(w, "w", _TYPES, index)
    if w.dim() != 2:
        raise ValueError("w must be taps x d")
    k = w.shape[0]
    _dense(w, "w", (k, d))
    if bias is not None:
        _device_tensor(bias, "bias", (w.dtype,), index)
        _dense(bias, "bias", (d,))
    if act not in ("none", "silu"):
        raise ValueError(f"act must be 'none' or 'silu', got {act!r}")
    states = (b, max(k - 1, 0), d)
    if s0 is not None:
        _device_tensor(s0, "s0", (x.dtype,), index)
        _dense(s0, "s0", states)
    _lengths(lengths, b, index)
    ys = (0, 0)
    if dy is not None:
        _device_tensor(dy, "dy", (x.dtype,), index)
        if dy.shape != x.shape:
            raise ValueError("dy and x disagree in shape")
        ys = _token_strides(dy, "dy")
    p = _CONV(b, n, d, *_token_strides(x, "x"), *ys, k, _DTYPE_CODE[x.dtype],
              _DTYPE_CODE[w.dtype], ACT[act])
    return p, index, states


def causal_conv(x: torch.Tensor, w: torch.Tensor, bias: Optional[torch.Tensor] = None,
                s0: Optional[torch.Tensor] = None, lengths: Optional[torch.Tensor] = None,
                act: str = "none", stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Short causal depthwise convolution over tokens: (y, s1).

    x: b x l x d (views with a dense last axis are read in place); w: taps x
    d, bias: d, of one dtype; s0: b x (taps - 1) x d of x's dtype, the inputs
    before the first token, or None for zeros; lengths: b int32 or None; act:
    'none' or 'silu'.  y: b x l x d of x's dtype, 0 past a length; s1: the
    last taps - 1 inputs."""
    p, index, states = _conv(x, w, bias, s0, lengths, act)
    with _on(index, stream):
        y = torch.empty_like(x, memory_format=_DENSE)
        s1 = x.new_empty(states)
        _raise(lib().dwc_causal_conv(p, x.data_ptr(), w.data_ptr(), _ptr(bias), _ptr(s0),
                                     _ptr(lengths), y.data_ptr(), s1.data_ptr(), _raw(index)))
    _returned(stream, index, y, s1)
    return y, s1


def causal_conv_step(x: torch.Tensor, w: torch.Tensor, bias: Optional[torch.Tensor] = None,
                     s0: Optional[torch.Tensor] = None, lengths: Optional[torch.Tensor] = None,
                     act: str = "none", out_state: Optional[torch.Tensor] = None, stream=None
                     ) -> Tuple[torch.Tensor, torch.Tensor]:
    """``causal_conv`` for one or a few new tokens of each sequence: (y, s1).
    out_state may be s0: the state is then updated in place."""
    p, index, states = _conv(x, w, bias, s0, lengths, act)
    if out_state is not None:
        _device_tensor(out_state, "out_state", (x.dtype,), index)
        _dense(out_state, "out_state", states)
    with _on(index, stream):
        y = torch.empty_like(x, memory_format=_DENSE)
        s1 = out_state
        if s1 is None:
            s1 = x.new_empty(states)
        _raise(lib().dwc_causal_conv_step(p, x.data_ptr(), w.data_ptr(), _ptr(bias), _ptr(s0),
                                          _ptr(lengths), y.data_ptr(), s1.data_ptr(),
                                          _raw(index)))
    _returned(stream, index, y, s1 if out_state is None else None)
    _written(out_state)
    return y, s1


def causal_conv_bwd(dy: torch.Tensor, ds1: Optional[torch.Tensor], x: torch.Tensor,
                    w: torch.Tensor, bias: Optional[torch.Tensor] = None,
                    s0: Optional[torch.Tensor] = None, lengths: Optional[torch.Tensor] = None,
                    act: str = "none", stream=None):
    """Gradients of ``causal_conv`` from those of y and s1 (None: zero):
    (dx, dw, dbias, ds0), dw and dbias fp32, dbias and ds0 None where bias
    and s0 are."""
    p, index, states = _conv(x, w, bias, s0, lengths, act, dy)
    if ds1 is not None:
        _device_tensor(ds1, "ds1", (x.dtype,), index)
        _dense(ds1, "ds1", states)
    with _on(index, stream):
        ws, need = _workspace(x, lib().dwc_causal_conv_bwd_workspace_size, p)
        dx = torch.empty_like(x, memory_format=_DENSE)
        dw = torch.empty_like(w, dtype=torch.float32)
        dbias = torch.empty_like(bias, dtype=torch.float32) if bias is not None else None
        ds0 = torch.empty_like(s0) if s0 is not None else None
        _raise(lib().dwc_causal_conv_bwd(p, dy.data_ptr(), _ptr(ds1), x.data_ptr(), w.data_ptr(),
                                         _ptr(bias), _ptr(s0), _ptr(lengths), dx.data_ptr(),
                                         dw.data_ptr(), _ptr(dbias), _ptr(ds0), ws.data_ptr(),
                                         need, _raw(index)))
    _returned(stream, index, dx, dw, dbias, ds0)
    return dx, dw, dbias, ds0


# ---------------------------------------------------------------- selective scan ----

def _scan(u, delta, A, B, C, D, z, delta_bias, s0, lengths, softplus, dy=None):
    """(the problem's bytes, device index, shape of the states)"""
    index = _device_tensor(u, "u", _TYPES)
    dt = (u.dtype,)
    shape = u.shape
    if len(shape) != 3:
        raise ValueError("u must be b x l x d")
    b, n, d = shape
    ds = _token_operand(delta, "delta", dt, index, shape)
    zs = _token_operand(z, "z", dt, index, shape) if z is not None else (0, 0)
    ys = _token_operand(dy, "dy", dt, index, shape) if dy is not None else (0, 0)
    _device_tensor(A, "A", _F32, index)
    if A.dim() != 2:
        raise ValueError("A must be d x n")
    m = A.shape[1]
    _dense(A, "A", (d, m))
    _device_tensor(B, "B", dt, index)
    _device_tensor(C, "C", dt, index)
    bs = B.shape
    if len(bs) != 4 or bs[0] != b or bs[1] != n or bs[3] != m or C.shape != bs:
        raise ValueError(f"B and C must be {(b, n, 'g', m)}")
    g = bs[2]
    if D is not None:
        _device_tensor(D, "D", _F32, index)
        _dense(D, "D", (d,))
    if delta_bias is not None:
        _device_tensor(delta_bias, "delta_bias", _F32, index)
        _dense(delta_bias, "delta_bias", (d,))
    states = (b, d, m)
    if s0 is not None:
        _device_tensor(s0, "s0", _F32, index)
        _dense(s0, "s0", states)
    _lengths(lengths, b, index)
    p = _SCAN(b, n, *_token_strides(u, "u"), *ds, *zs, *ys, *_strides(B, "B"),
              *_strides(C, "C"), d, m, g, _DTYPE_CODE[u.dtype], int(bool(softplus)), 0)
    return p, index, states


def selective_scan_step(u: torch.Tensor, delta: torch.Tensor, A: torch.Tensor, B: torch.Tensor,
                        C: torch.Tensor, D: Optional[torch.Tensor] = None,
                        z: Optional[torch.Tensor] = None,
                        delta_bias: Optional[torch.Tensor] = None,
                        s0: Optional[torch.Tensor] = None,
                        lengths: Optional[torch.Tensor] = None, softplus: bool = False,
                        out_state: Optional[torch.Tensor] = None, stream=None
                        ) -> Tuple[torch.Tensor, torch.Tensor]:
    """The selective scan token by token: (y, s1).  The form for one or a few
    new tokens of each sequence; shapes as ``selective_scan``.  out_state may
    be s0: the state is then updated in place."""
    p, index, states = _scan(u, delta, A, B, C, D, z, delta_bias, s0, lengths, softplus)
    if out_state is not None:
        _device_tensor(out_state, "out_state", _F32, index)
        _dense(out_state, "out_state", states)
    with _on(index, stream):
        y = torch.empty_like(u, memory_format=_DENSE)
        s1 = out_state
        if s1 is None:
            s1 = A.new_empty(states)
        _raise(lib().dwc_scan_step(p, u.data_ptr(), delta.data_ptr(), A.data_ptr(), B.data_ptr(),
                                   C.data_ptr(), _ptr(D), _ptr(z), _ptr(delta_bias), _ptr(s0),
                                   _ptr(lengths), y.data_ptr(), s1.data_ptr(), _raw(index)))
    _returned(stream, index, y, s1 if out_state is None else None)
    _written(out_state)
    return y, s1


def selective_scan(u: torch.Tensor, delta: torch.Tensor, A: torch.Tensor, B: torch.Tensor,
                   C: torch.Tensor, D: Optional[torch.Tensor] = None,
                   z: Optional[torch.Tensor] = None, delta_bias: Optional[torch.Tensor] = None,
                   s0: Optional[torch.Tensor] = None, lengths: Optional[torch.Tensor] = None,
                   softplus: bool = False, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """The selective state space scan over whole sequences: (y, s1).

    u, delta, z: b x l x d; B, C: b x l x g x n, shared by the d / g channels
    of a group (views with a dense last axis are read in place); A: d x n
    fp32, D, delta_bias: d fp32; s0: b x d x n fp32 or None; lengths: b int32
    or None.  The steps are delta + delta_bias, with ``softplus`` their
    softplus.  y: b x l x d of u's dtype; s1: the states after the last
    token."""
    p, index, states = _scan(u, delta, A, B, C, D, z, delta_bias, s0, lengths, softplus)
    with _on(index, stream):
        ws, need = _workspace(u, lib().dwc_scan_workspace_size, p, SCAN_FWD)
        y = torch.empty_like(u, memory_format=_DENSE)
        s1 = A.new_empty(states)
        _raise(lib().dwc_scan_fwd(p, u.data_ptr(), delta.data_ptr(), A.data_ptr(), B.data_ptr(),
                                  C.data_ptr(), _ptr(D), _ptr(z), _ptr(delta_bias), _ptr(s0),
                                  _ptr(lengths), y.data_ptr(), s1.data_ptr(), ws.data_ptr(), need,
                                  _raw(index)))
    _returned(stream, index, y, s1)
    return y, s1


def selective_scan_bwd(dy: torch.Tensor, ds1: Optional[torch.Tensor], u: torch.Tensor,
                       delta: torch.Tensor, A: torch.Tensor, B: torch.Tensor, C: torch.Tensor,
                       D: Optional[torch.Tensor] = None, z: Optional[torch.Tensor] = None,
                       delta_bias: Optional[torch.Tensor] = None,
                       s0: Optional[torch.Tensor] = None,
                       lengths: Optional[torch.Tensor] = None, softplus: bool = False,
                       stream=None):
    """Gradients of ``selective_scan`` from those of y and s1 (None: zero):
    (du, ddelta, dA, dB, dC, dD, dz, ddelta_bias, ds0), None where the
    argument is.  dA, dD, ddelta_bias and ds0 are fp32."""
    p, index, states = _scan(u, delta, A, B, C, D, z, delta_bias, s0, lengths, softplus, dy)
    if ds1 is not None:
        _device_tensor(ds1, "ds1", _F32, index)
        _dense(ds1, "ds1", states)
    like = lambda t: torch.empty_like(t, memory_format=_DENSE) if t is not None else None  # noqa: E731
    with _on(index, stream):
        ws, need = _workspace(u, lib().dwc_scan_workspace_size, p, SCAN_BWD)
        du, ddelta, dA, dB, dC, dD, dz, dbias, ds0 = map(like, (u, delta, A, B, C, D, z,
                                                                delta_bias, s0))
        _raise(lib().dwc_scan_bwd(p, dy.data_ptr(), _ptr(ds1), u.data_ptr(), delta.data_ptr(),
                                  A.data_ptr(), B.data_ptr(), C.data_ptr(), _ptr(D), _ptr(z),
                                  _ptr(delta_bias), _ptr(s0), _ptr(lengths), du.data_ptr(),
                                  ddelta.data_ptr(), dA.data_ptr(), dB.data_ptr(), dC.data_ptr(),
                                  _ptr(dD), _ptr(dz), _ptr(dbias), _ptr(ds0), ws.data_ptr(), need,
                                  _raw(index)))
    _returned(stream, index, du, ddelta, dA, dB, dC, dD, dz, dbias, ds0)
    return du, ddelta, dA, dB, dC, dD, dz, dbias, ds0


# ----------------------------------------------------------------- residual norm ----

def _row_operand(t, name, dtypes, index, shape):
    """Its row stride, checked against the block's output."""
    _device_tensor(t, name, dtypes, index)
    if t.shape != shape:
        raise ValueError(f"{name} and y disagree in shape")
    return _row_stride(t, name)


def _resnorm(x, y, gate, scale, w_post, w_pre, post, pre, act, eps, dr=None, dh=None):
    """(the problem's bytes, device index)"""
    index = _device_tensor(y, "y", _TYPES)
    shape = y.shape
    if len(shape) < 1 or shape[-1] < 1:
        raise ValueError("y needs a last axis of at least one element")
    c = shape[-1]
    xt = y.dtype if x is None else x.dtype
    if dr is not None and x is None:
        xt = dr.dtype
    yt = (y.dtype,)
    strides = (_row_operand(x, "x", (torch.float32, y.dtype), index, shape) if x is not None else c,
               _row_stride(y, "y"),
               _row_operand(gate, "gate", yt, index, shape) if gate is not None else c,
               _row_operand(dr, "dr", (xt,), index, shape) if dr is not None else c,
               _row_operand(dh, "dh", yt, index, shape) if dh is not None else c)
    wt = None
    for t, name in ((scale, "scale"), (w_post, "w_post"), (w_pre, "w_pre")):
        if t is not None:
            _device_tensor(t, name, _TYPES if wt is None else (wt,), index)
            _dense(t, name, (c,))
            wt = t.dtype
    if act not in GATE:
        raise ValueError(f"act must be one of {sorted(GATE)}, got {act!r}")
    if (w_post is not None and not post) or (w_pre is not None and not pre):
        raise ValueError("weights are not given without their norm")
    p = _RESNORM(y.numel() // c, c, *strides, _DTYPE_CODE[xt], _DTYPE_CODE[y.dtype],
                 _DTYPE_CODE[wt] if wt is not None else 0, GATE[act], int(bool(post)),
                 int(bool(pre)), eps, 0)
    return p, index


def residual_norm(x: Optional[torch.Tensor], y: torch.Tensor,
                  gate: Optional[torch.Tensor] = None, scale: Optional[torch.Tensor] = None,
                  w_post: Optional[torch.Tensor] = None, w_pre: Optional[torch.Tensor] = None,
                  eps: float = 1e-5, post: bool = True, pre: bool = True, act: str = "none",
                  stream=None):
    """r = x + scale act(gate) norm(y) w_post and h = norm(r) w_pre over the
    last axis, norm(v) = v / sqrt(mean(v^2) + eps): (r, h, post_rstd,
    pre_rstd), the last two 1 / sqrt(...) of y and r, fp32, one a row.

    x: the residual, fp32 or of y's dtype, or None for zeros (r is then of
    y's dtype); gate: of y's shape and dtype, act 'none', 'silu' or 'sigmoid';
    scale, w_post, w_pre: of the last axis, one dtype.  Without ``post`` y is
    not normalised, without ``pre`` h and pre_rstd are None."""
    p, index = _resnorm(x, y, gate, scale, w_post, w_pre, post, pre, act, eps)
    with _on(index, stream):
        r = torch.empty_like(y if x is None else x, memory_format=_DENSE)
        h = torch.empty_like(y, memory_format=_DENSE) if pre else None
        q1 = y.new_empty(y.shape[:-1], dtype=torch.float32) if post else None
        q2 = None
        if pre:
            q2 = torch.empty_like(q1) if post else y.new_empty(y.shape[:-1], dtype=torch.float32)
        _raise(lib().dwc_residual_norm(p, _ptr(x), y.data_ptr(), _ptr(gate), _ptr(scale),
                                       _ptr(w_post), _ptr(w_pre), r.data_ptr(), _ptr(h), _ptr(q1),
                                       _ptr(q2), _raw(index)))
    _returned(stream, index, r, h, q1, q2)
    return r, h, q1, q2


def residual_norm_bwd(dr: Optional[torch.Tensor], dh: Optional[torch.Tensor],
                      x: Optional[torch.Tensor], y: torch.Tensor,
                      post_rstd: Optional[torch.Tensor], pre_rstd: Optional[torch.Tensor],
                      gate: Optional[torch.Tensor] = None, scale: Optional[torch.Tensor] = None,
                      w_post: Optional[torch.Tensor] = None,
                      w_pre: Optional[torch.Tensor] = None, post: bool = True, pre: bool = True,
                      act: str = "none", stream=None):
    """Gradients of ``residual_norm`` from those of r and h (one may be None
    for zero): (dx, dy, dgate, dscale, dw_post, dw_pre), None where the
    argument is; dscale, dw_post and dw_pre are fp32."""
    if dr is None and dh is None:
        raise ValueError("dr or dh must be given")
    if dh is not None and not pre:
        raise ValueError("dh is not given without pre")
    p, index = _resnorm(x, y, gate, scale, w_post, w_pre, post, pre, act, 0.0, dr, dh)
    for t, name, need in ((post_rstd, "post_rstd", post), (pre_rstd, "pre_rstd", dh is not None)):
        if t is not None or need:
            _device_tensor(t, name, _F32, index)
            _dense(t, name, y.shape[:-1])
    with _on(index, stream):
        ws, need = _workspace(y, lib().dwc_residual_norm_bwd_workspace_size, p)
        dx = torch.empty_like(x, memory_format=_DENSE) if x is not None else None
        dy = torch.empty_like(y, memory_format=_DENSE)
        dgate = torch.empty_like(y, memory_format=_DENSE) if gate is not None else None
        sums = [torch.empty_like(t, dtype=torch.float32) if t is not None else None
                for t in (scale, w_post, w_pre)]
        _raise(lib().dwc_residual_norm_bwd(p, _ptr(dr), _ptr(dh), _ptr(x), y.data_ptr(),
                                           _ptr(post_rstd), _ptr(pre_rstd), _ptr(gate),
                                           _ptr(scale), _ptr(w_post), _ptr(w_pre), _ptr(dx),
                                           dy.data_ptr(), _ptr(dgate), *map(_ptr, sums),
                                           ws.data_ptr(), need, _raw(index)))
    _returned(stream, index, dx, dy, dgate, *sums)
    return (dx, dy, dgate, *sums)


__all__ = ["causal_conv", "causal_conv_step", "causal_conv_bwd", "selective_scan",
           "selective_scan_step", "selective_scan_bwd", "residual_norm", "residual_norm_bwd",
           "CausalConvProblem", "ScanProblem", "ResNormProblem", "SCAN_FWD", "SCAN_BWD", "GATE"]
