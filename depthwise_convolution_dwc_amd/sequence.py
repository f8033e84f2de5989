"""Operators of the sequence layer around a depthwise convolution: layer
norm, dropout from a counter-based generator and the gated delta rule, on
torch tensors.  Argument marshalling only, like the package's other calls;
the formulas stand in include/dwc.h.

Every call runs on the current stream of the tensors' device, or on
``stream``.  What a call allocates comes from the memory of the stream that
it runs on, and outputs are recorded on the current one too, so that the
allocator does not hand a block out while either stream has work on it; the
caller orders the two streams' work on the tensors themselves.
"""

from __future__ import annotations

import contextlib
import ctypes
import math
import struct
from typing import Optional, Tuple, Union

import torch

from . import _DTYPE_CODE, _raise, lib

DELTA_FWD, DELTA_BWD = 0, 1
_TYPES = (torch.float32, torch.bfloat16, torch.float16)
_F32, _I32 = (torch.float32,), (torch.int32,)
_I3 = ctypes.c_int64 * 3
_DENSE = torch.contiguous_format


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


# The problems as the calls below pass them: the structures' bytes, packed in
# one step (a small call costs the host about as long as the kernel runs).
_NORM = struct.Struct("4q3if").pack
_DROPOUT = struct.Struct("qdQQ2i").pack
_DELTA = struct.Struct("20q5if").pack


def bind(l: ctypes.CDLL) -> None:
    """Argument types of the sequence-layer entry points; a problem may be
    passed by reference or as the structure's bytes."""
    vp, sz = ctypes.c_void_p, ctypes.c_size_t
    l.dwc_layer_norm.argtypes = [vp] * 8
    l.dwc_layer_norm_bwd_workspace_size.argtypes = [vp, ctypes.POINTER(sz)]
    l.dwc_layer_norm_bwd.argtypes = [vp] * 10 + [sz, vp]
    l.dwc_dropout.argtypes = [vp] * 5
    l.dwc_dropout_at.argtypes = [vp] * 6
    l.dwc_delta_step.argtypes = [vp] * 11
    l.dwc_delta_workspace_size.argtypes = [vp, ctypes.c_int, ctypes.POINTER(sz)]
    l.dwc_delta_fwd.argtypes = [vp] * 11 + [sz, vp]
    l.dwc_delta_bwd.argtypes = [vp] * 17 + [sz, vp]


_HERE = contextlib.nullcontext()


def _on(index, stream):
    """The device made current, if it is not; with a stream given, that
    stream."""
    if stream is None:
        return _HERE if index == torch._C._cuda_getDevice() else torch.cuda.device(index)
    if not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(int(stream), device=index)
    if stream.device_index != index:
        raise ValueError(f"stream must be one of cuda:{index}, got cuda:{stream.device_index}")
    return torch.cuda.stream(stream)


def _raw(index):
    """The current stream's handle."""
    return torch._C._cuda_getCurrentRawStream(index)


def _returned(stream, index, *made):
    """Tensors allocated on a stream given are marked as used on the current
    one, where the caller drops them."""
    if stream is not None:
        here = torch.cuda.current_stream(index)
        for t in made:
            if t is not None:
                t.record_stream(here)


def _written(t):
    """A tensor that was given to be written: graphs that saved it know."""
    if t is not None and not t.is_inference():
        torch.autograd.graph.increment_version(t)


def _device_tensor(t, name, dtypes, index=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    at = t.get_device()
    if at < 0 or not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if index is not None and at != index:
        raise ValueError(f"{name} must be on cuda:{index}, got {t.device}")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must be one of {dtypes}, got {t.dtype}")
    return at


def _dense(t, name, shape):
    if t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous of shape {tuple(shape)}, "
                         f"got {tuple(t.shape)}")


def _ptr(t):
    return t.data_ptr() if t is not None else None


def _row_stride(t, name):
    """Elements between the rows of (..., c) seen as rows x c; raises where
    the leading axes do not form one stride or the last is not dense."""
    c = t.shape[-1]
    if t.is_contiguous() or t.numel() == 0:
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


def _weights(w, b, c, index):
    for t, name in ((w, "w"), (b, "b")):
        if t is not None:
            _device_tensor(t, name, _TYPES, index)
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
    index = _device_tensor(x, "x", _TYPES)
    shape = x.shape
    if len(shape) < 1 or shape[-1] < 1:
        raise ValueError("x needs a last axis of at least one element")
    c, lead = shape[-1], shape[:-1]
    wt = _weights(w, b, c, index)
    if out is not None:
        _device_tensor(out, "out", _TYPES if out_dtype is None else (out_dtype,), index)
        _dense(out, "out", shape)
        out_dtype = out.dtype
    out_dtype = out_dtype or x.dtype
    if out_dtype not in _TYPES:
        raise TypeError(f"out_dtype must be one of {_TYPES}, got {out_dtype}")
    p = _NORM(x.numel() // c, c, _row_stride(x, "x"), c, _DTYPE_CODE[x.dtype],
              _DTYPE_CODE[out_dtype], wt, eps)
    with _on(index, stream):
        y = out
        if y is None:
            y = torch.empty_like(x, dtype=out_dtype, memory_format=_DENSE)
        mean = x.new_empty(lead, dtype=torch.float32)
        rstd = torch.empty_like(mean)
        _raise(lib().dwc_layer_norm(p, x.data_ptr(), _ptr(w), _ptr(b), y.data_ptr(),
                                    mean.data_ptr(), rstd.data_ptr(), _raw(index)))
    _returned(stream, index, y if out is None else None, mean, rstd)
    _written(out)
    return y, mean, rstd


def layer_norm_bwd(dy: torch.Tensor, x: torch.Tensor, mean: torch.Tensor, rstd: torch.Tensor,
                   w: Optional[torch.Tensor] = None, stream=None
                   ) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """Gradients of ``layer_norm``: (dx of x's dtype, dw, db fp32)."""
    index = _device_tensor(x, "x", _TYPES)
    _device_tensor(dy, "dy", _TYPES, index)
    shape = x.shape
    if dy.shape != shape:
        raise ValueError("dy and x disagree in shape")
    if len(shape) < 1 or shape[-1] < 1:
        raise ValueError("x needs a last axis of at least one element")
    c, lead = shape[-1], shape[:-1]
    for t, name in ((mean, "mean"), (rstd, "rstd")):
        _device_tensor(t, name, _F32, index)
        _dense(t, name, lead)
    wt = _weights(w, None, c, index)
    p = _NORM(x.numel() // c, c, _row_stride(x, "x"), _row_stride(dy, "dy"),
              _DTYPE_CODE[x.dtype], _DTYPE_CODE[dy.dtype], wt, 0.0)
    with _on(index, stream):
        need = ctypes.c_size_t()
        _raise(lib().dwc_layer_norm_bwd_workspace_size(p, ctypes.byref(need)))
        ws = x.new_empty(need.value, dtype=torch.uint8)
        dx = torch.empty_like(x, memory_format=_DENSE)
        dw = x.new_empty(c, dtype=torch.float32)
        db = torch.empty_like(dw)
        _raise(lib().dwc_layer_norm_bwd(p, dy.data_ptr(), x.data_ptr(), mean.data_ptr(),
                                        rstd.data_ptr(), _ptr(w), dx.data_ptr(), dw.data_ptr(),
                                        db.data_ptr(), ws.data_ptr(), need.value,
                                        _raw(index)))
    _returned(stream, index, dx, dw, db)
    return dx, dw, db


def dropout(x: torch.Tensor, p: float, seed: int, offset: Union[int, torch.Tensor] = 0,
            residual: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
            stream=None) -> torch.Tensor:
    """residual + (kept ? x / (1 - p) : 0), the mask a function of (seed,
    offset, element index).  The gradient of x is this call on dy with the
    same p, seed and offset; elements of later calls that must not share a
    mask take an offset at least (numel + 3) // 4 further.  An offset may be
    one int64 value in device memory, which is read when the kernel runs: a
    captured call then takes a new one with each replay."""
    index = _device_tensor(x, "x", _TYPES)
    if not x.is_contiguous():
        raise ValueError("x must be contiguous")
    if residual is not None:
        _device_tensor(residual, "residual", (x.dtype,), index)
        _dense(residual, "residual", x.shape)
    at = None
    if isinstance(offset, torch.Tensor):
        at, offset = offset, 0
        _device_tensor(at, "offset", (torch.int64,), index)
        if at.numel() != 1:
            raise ValueError("offset must be one value")
    if not 0 <= int(seed) < 1 << 64 or not 0 <= int(offset) < 1 << 64:
        raise ValueError("seed and offset must be in 0 .. 2^64 - 1")
    if out is not None:
        _device_tensor(out, "out", (x.dtype,), index)
        _dense(out, "out", x.shape)
    d = _DROPOUT(x.numel(), p, int(seed), int(offset), _DTYPE_CODE[x.dtype], 0)
    with _on(index, stream):
        y = out
        if y is None:
            y = torch.empty_like(x, memory_format=_DENSE)
        s = _raw(index)
        if at is None:
            _raise(lib().dwc_dropout(d, x.data_ptr(), _ptr(residual), y.data_ptr(), s))
        else:
            _raise(lib().dwc_dropout_at(d, x.data_ptr(), _ptr(residual), y.data_ptr(),
                                        at.data_ptr(), s))
    _returned(stream, index, y if out is None else None)
    _written(out)
    return y


def _strides(t, name):
    """(batch, token, head) strides of a b x l x h x d tensor."""
    s = t.stride()
    if s[3] != 1 and t.shape[3] > 1 and t.numel():
        raise ValueError(f"{name}'s last axis must be dense")
    return s[:3]


def _delta(q, k, v, g, beta, s0, lengths, scale, dout=None):
    """(the problem's bytes, device index, shape of the states)"""
    index = _device_tensor(q, "q", _TYPES)
    dt = (q.dtype,)
    _device_tensor(k, "k", dt, index)
    _device_tensor(v, "v", dt, index)
    _device_tensor(g, "g", _F32, index)
    _device_tensor(beta, "beta", _F32, index)
    shape = q.shape
    if len(shape) != 4 or v.dim() != 4:
        raise ValueError("q, k and v must be b x l x heads x head size")
    b, n, hk, dk = shape
    vb, vn, hv, dv = v.shape
    if k.shape != shape or vb != b or vn != n:
        raise ValueError("q, k and v disagree in shape")
    if g.shape != (b, n, hv) or beta.shape != (b, n, hv):
        raise ValueError(f"g and beta must be {(b, n, hv)}")
    states = (b, hv, dk, dv)
    if s0 is not None:
        _device_tensor(s0, "s0", _F32, index)
        _dense(s0, "s0", states)
    if lengths is not None:
        _device_tensor(lengths, "lengths", _I32, index)
        _dense(lengths, "lengths", (b,))
    do = (0, 0, 0)
    if dout is not None:
        _device_tensor(dout, "dout", dt, index)
        if dout.shape != v.shape:
            raise ValueError("dout and v disagree in shape")
        do = _strides(dout, "dout")
    if scale is None:
        scale = 1.0 / math.sqrt(dk) if dk else 1.0
    p = _DELTA(b, n, *_strides(q, "q"), *_strides(k, "k"), *_strides(v, "v"), *g.stride(),
               *beta.stride(), *do, hk, hv, dk, dv, _DTYPE_CODE[q.dtype], scale)
    return p, index, states


def _workspace(p, op, like):
    need = ctypes.c_size_t()
    _raise(lib().dwc_delta_workspace_size(p, op, ctypes.byref(need)))
    return like.new_empty(need.value, dtype=torch.uint8), need.value


def delta_rule_step(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, g: torch.Tensor,
                    beta: torch.Tensor, s0: Optional[torch.Tensor] = None,
                    lengths: Optional[torch.Tensor] = None, scale: Optional[float] = None,
                    out_state: Optional[torch.Tensor] = None, stream=None
                    ) -> Tuple[torch.Tensor, torch.Tensor]:
    """The gated delta rule token by token: (o, s1).  The form for one or a
    few new tokens of each sequence; shapes as ``delta_rule``.  out_state
    may be s0: the state is then updated in place."""
    p, index, states = _delta(q, k, v, g, beta, s0, lengths, scale)
    if out_state is not None:
        _device_tensor(out_state, "out_state", _F32, index)
        _dense(out_state, "out_state", states)
    with _on(index, stream):
        o = torch.empty_like(v, memory_format=_DENSE)
        s1 = out_state
        if s1 is None:
            s1 = g.new_empty(states)
        _raise(lib().dwc_delta_step(p, q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(),
                                    beta.data_ptr(), _ptr(s0), _ptr(lengths), o.data_ptr(),
                                    s1.data_ptr(), _raw(index)))
    _returned(stream, index, o, s1 if out_state is None else None)
    _written(out_state)
    return o, s1


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
    p, index, states = _delta(q, k, v, g, beta, s0, lengths, scale)
    with _on(index, stream):
        ws, need = _workspace(p, DELTA_FWD, q)
        o = torch.empty_like(v, memory_format=_DENSE)
        s1 = g.new_empty(states)
        _raise(lib().dwc_delta_fwd(p, q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(),
                                   beta.data_ptr(), _ptr(s0), _ptr(lengths), o.data_ptr(),
                                   s1.data_ptr(), ws.data_ptr(), need, _raw(index)))
    _returned(stream, index, o, s1)
    return o, s1


def delta_rule_bwd(dout: torch.Tensor, ds1: Optional[torch.Tensor], q: torch.Tensor,
                   k: torch.Tensor, v: torch.Tensor, g: torch.Tensor, beta: torch.Tensor,
                   s0: Optional[torch.Tensor] = None, lengths: Optional[torch.Tensor] = None,
                   scale: Optional[float] = None, stream=None):
    """Gradients of ``delta_rule`` from those of o and s1 (None: zero):
    (dq, dk, dv, dg, dbeta, ds0), ds0 None where s0 is."""
    p, index, states = _delta(q, k, v, g, beta, s0, lengths, scale, dout)
    if ds1 is not None:
        _device_tensor(ds1, "ds1", _F32, index)
        _dense(ds1, "ds1", states)
    with _on(index, stream):
        ws, need = _workspace(p, DELTA_BWD, q)
        dq = torch.empty_like(q, memory_format=_DENSE)
        dk = torch.empty_like(q, memory_format=_DENSE)
        dv = torch.empty_like(v, memory_format=_DENSE)
        dg = torch.empty_like(g, memory_format=_DENSE)
        dbeta = torch.empty_like(g, memory_format=_DENSE)
        ds0 = torch.empty_like(s0) if s0 is not None else None
        _raise(lib().dwc_delta_bwd(p, dout.data_ptr(), _ptr(ds1), q.data_ptr(), k.data_ptr(),
                                   v.data_ptr(), g.data_ptr(), beta.data_ptr(), _ptr(s0),
                                   _ptr(lengths), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(),
                                   dg.data_ptr(), dbeta.data_ptr(), _ptr(ds0), ws.data_ptr(),
                                   need, _raw(index)))
    _returned(stream, index, dq, dk, dv, dg, dbeta, ds0)
    return dq, dk, dv, dg, dbeta, ds0


__all__ = ["layer_norm", "layer_norm_bwd", "dropout", "delta_rule", "delta_rule_step",
           "delta_rule_bwd", "NormProblem", "DropoutProblem", "DeltaProblem", "DELTA_FWD",
           "DELTA_BWD"]
