"""PyTorch autograd wrapper of libdwc: a depthwise Conv2d whose forward,
data gradient and filter gradient all run in libdwc's HIP kernels.

Layouts follow the library (Flash-DWC, TACO, §2.3: channel-last tensors):
activations N x H x W x C and the filter FH x FW x C.  A module stores its
weight in that FH x FW x C layout, so a training step moves no weights
around; ``weight_from_torch`` / ``weight_to_torch`` convert from / to the
C x 1 x FH x FW layout of ``torch.nn.Conv2d(groups=C)``.

Inputs may be given channel-last (``layout="nhwc"``, a contiguous
N x H x W x C tensor) or as logical NCHW tensors in ``torch.channels_last``
memory format (``layout="nchw"``), whose memory already is N x H x W x C:
both are passed to the library without a copy.  A logical NCHW tensor in
another memory format is made channels_last first (one copy).

Outputs and gradients are computed in fp32 (the library's output type).  For
bf16/fp16 operands the forward returns fp32; the backward rounds the
incoming gradient to the operand dtype (the library takes X, W and dY in one
dtype) and returns dX and dW in the dtypes of X and W.

Layer norm, dropout and the gated delta rule have autograd wrappers here too,
and ``GatedDeltaMixer`` is the sequence layer that runs them together with a
causal depthwise convolution.  So have the short causal convolution over
tokens, the selective scan and the residual norm; ``SelectiveScanMixer`` and
``SelectiveScanLayers`` run those together.
"""

from __future__ import annotations

import functools
import itertools
import math
from typing import List, NamedTuple, Optional, Tuple, Union

import torch
import torch.nn.functional as F

from . import bwd_data, bwd_filter, fwd, sequence, space

IntPair = Union[int, Tuple[int, int]]


def _pair(v: IntPair) -> Tuple[int, int]:
    if isinstance(v, (tuple, list)):
        return int(v[0]), int(v[1])
    return int(v), int(v)


def weight_from_torch(w: torch.Tensor) -> torch.Tensor:
    """C x 1 x FH x FW (torch.nn.Conv2d, groups = C) -> FH x FW x C, contiguous."""
    if w.dim() != 4 or w.shape[1] != 1:
        raise ValueError(f"expected a C x 1 x FH x FW depthwise weight, got {tuple(w.shape)}")
    return w[:, 0].permute(1, 2, 0).contiguous()


def weight_to_torch(w: torch.Tensor) -> torch.Tensor:
    """FH x FW x C -> C x 1 x FH x FW (torch.nn.Conv2d, groups = C), contiguous."""
    if w.dim() != 3:
        raise ValueError(f"expected an FH x FW x C weight, got {tuple(w.shape)}")
    return w.permute(2, 0, 1).unsqueeze(1).contiguous()


def _to_nhwc(x: torch.Tensor, layout: str) -> torch.Tensor:
    if layout == "nhwc":
        return x.contiguous()
    if layout == "nchw":
        if x.dim() != 4:
            raise ValueError(f"expected a 4-d NCHW tensor, got {tuple(x.shape)}")
        return x.contiguous(memory_format=torch.channels_last).permute(0, 2, 3, 1)
    raise ValueError(f"layout must be 'nhwc' or 'nchw', got {layout!r}")


def _from_nhwc(y: torch.Tensor, layout: str) -> torch.Tensor:
    # an N x H x W x C tensor seen as logical NCHW in channels_last memory
    return y if layout == "nhwc" else y.permute(0, 3, 1, 2)


class DepthwiseConv2dFunction(torch.autograd.Function):
    """Y = DWC(X, W) on channel-last tensors (X: N x H x W x C, W: FH x FW x C).

    forward: ``dwc_fwd``; backward: ``dwc_bwd_data`` for dX and
    ``dwc_bwd_filter`` for dW (Flash-DWC §5.1), at any stride and padding."""

    @staticmethod
    def forward(ctx, x: torch.Tensor, w: torch.Tensor, stride: Tuple[int, int],
                pad: Tuple[int, int], algo: str) -> torch.Tensor:
        ctx.save_for_backward(x, w)
        ctx.stride, ctx.pad, ctx.algo = stride, pad, algo
        return fwd(x, w, stride, pad, algo=algo)

    @staticmethod
    def backward(ctx, gy: torch.Tensor):
        x, w = ctx.saved_tensors
        gy = gy.to(x.dtype).contiguous()
        dx = dw = None
        if ctx.needs_input_grad[0]:
            dx = bwd_data(gy, w, (x.shape[1], x.shape[2]), ctx.stride, ctx.pad, algo=ctx.algo)
            dx = dx.to(x.dtype)
        if ctx.needs_input_grad[1]:
            dw = bwd_filter(x, gy, (w.shape[0], w.shape[1]), ctx.stride, ctx.pad, algo=ctx.algo)
            dw = dw.to(w.dtype)
        return dx, dw, None, None, None


def depthwise_conv2d(x: torch.Tensor, weight: torch.Tensor, stride: IntPair = 1,
                     padding: IntPair = 0, layout: str = "nhwc",
                     algo: str = "auto") -> torch.Tensor:
    """Depthwise 2-D cross-correlation with autograd.

    x: N x H x W x C (``layout="nhwc"``) or logical N x C x H x W
    (``layout="nchw"``); weight: FH x FW x C.  Returns fp32 in the same
    layout as x."""
    if weight.dim() != 3:
        raise ValueError(f"weight must be FH x FW x C, got {tuple(weight.shape)}")
    xn = _to_nhwc(x, layout)
    y = DepthwiseConv2dFunction.apply(xn, weight.contiguous(), _pair(stride), _pair(padding),
                                      algo)
    return _from_nhwc(y, layout)


class DepthwiseConv2d(torch.nn.Module):
    """Depthwise Conv2d (groups = channels, no bias) on libdwc.

    The weight parameter is FH x FW x C.  Initialised like torch.nn.Conv2d:
    uniform in +-1/sqrt(FH * FW) (kaiming-uniform with a = sqrt(5) for a
    fan-in of FH * FW)."""

    def __init__(self, channels: int, kernel_size: IntPair, stride: IntPair = 1,
                 padding: IntPair = 0, layout: str = "nchw", algo: str = "auto",
                 device=None, dtype=torch.float32):
        super().__init__()
        if layout not in ("nhwc", "nchw"):
            raise ValueError(f"layout must be 'nhwc' or 'nchw', got {layout!r}")
        self.channels = int(channels)
        self.kernel_size = _pair(kernel_size)
        self.stride = _pair(stride)
        self.padding = _pair(padding)
        self.layout = layout
        self.algo = algo
        fh, fw = self.kernel_size
        self.weight = torch.nn.Parameter(torch.empty((fh, fw, self.channels), device=device,
                                                     dtype=dtype))
        bound = 1.0 / math.sqrt(fh * fw)
        with torch.no_grad():
            self.weight.uniform_(-bound, bound)

    @classmethod
    def from_torch(cls, conv: torch.nn.Conv2d, layout: str = "nchw", algo: str = "auto"):
        """A module with the weights of a depthwise torch.nn.Conv2d (no bias,
        no dilation, zero padding given as numbers)."""
        c = conv.in_channels
        if conv.groups != c or conv.out_channels != c or conv.bias is not None:
            raise ValueError("need groups == in_channels == out_channels and no bias")
        if tuple(conv.dilation) != (1, 1) or isinstance(conv.padding, str) \
                or conv.padding_mode != "zeros":
            raise ValueError("need dilation 1 and numeric zero padding")
        m = cls(c, conv.kernel_size, conv.stride, conv.padding, layout, algo,
                device=conv.weight.device, dtype=conv.weight.dtype)
        with torch.no_grad():
            m.weight.copy_(weight_from_torch(conv.weight))
        return m

    def torch_weight(self) -> torch.Tensor:
        """The weight in torch.nn.Conv2d's C x 1 x FH x FW layout (a copy)."""
        return weight_to_torch(self.weight.detach())

    def forward(self, x: torch.Tensor) -> torch.Tensor:
        return depthwise_conv2d(x, self.weight, self.stride, self.padding, self.layout,
                                self.algo)

    def extra_repr(self) -> str:
        return (f"{self.channels}, kernel_size={self.kernel_size}, stride={self.stride}, "
                f"padding={self.padding}, layout={self.layout!r}")


class _Gradients(torch.autograd.Function):
    """A call that makes gradients and has none of its own: a second
    derivative that needs them raises, on whatever path it comes."""

    @staticmethod
    def forward(ctx, call, *tensors):
        return call(*tensors)

    @staticmethod
    def backward(ctx, *grads):
        raise RuntimeError("layer_norm, delta_rule, causal_conv, selective_scan and "
                           "residual_norm are differentiable once")


def _gradients(call, *tensors):
    return _Gradients.apply(call, *tensors) if torch.is_grad_enabled() else call(*tensors)


class LayerNormFunction(torch.autograd.Function):
    """``sequence.layer_norm`` and its gradients; mean and rstd are kept, the
    normalised rows are computed again.  Differentiable once."""

    @staticmethod
    def forward(ctx, x, w, b, eps, out_dtype):
        y, mean, rstd = sequence.layer_norm(x, w, b, eps, out_dtype)
        ctx.save_for_backward(x, w, mean, rstd)
        ctx.b_dtype = b.dtype if b is not None else None
        return y

    @staticmethod
    def backward(ctx, gy):
        x, w, mean, rstd = ctx.saved_tensors
        dx, dw, db = _gradients(sequence.layer_norm_bwd, gy.contiguous(), x, mean, rstd, w)
        return (dx, dw.to(w.dtype) if w is not None else None,
                db.to(ctx.b_dtype) if ctx.b_dtype is not None else None, None, None)


def layer_norm(x: torch.Tensor, w: Optional[torch.Tensor] = None,
               b: Optional[torch.Tensor] = None, eps: float = 1e-5,
               out_dtype: Optional[torch.dtype] = None) -> torch.Tensor:
    """Layer norm over the last axis with autograd; y is of ``out_dtype`` (x's
    by default).  A matrix with a row stride is read in place; other views
    are made contiguous first (one copy)."""
    if x.dim() != 2 or x.stride(1) != 1 or x.stride(0) < x.shape[1]:
        x = x.contiguous()
    return LayerNormFunction.apply(x, w, b, eps, out_dtype)


class LayerNorm(torch.nn.Module):
    """Layer norm over the last axis; weight and bias fp32 unless ``dtype``
    says otherwise."""

    def __init__(self, channels: int, eps: float = 1e-5, bias: bool = True, device=None,
                 dtype=torch.float32):
        super().__init__()
        self.channels, self.eps = int(channels), float(eps)
        self.weight = torch.nn.Parameter(torch.ones(self.channels, device=device, dtype=dtype))
        self.bias = torch.nn.Parameter(
            torch.zeros(self.channels, device=device, dtype=dtype)) if bias else None

    def forward(self, x: torch.Tensor, out_dtype: Optional[torch.dtype] = None) -> torch.Tensor:
        return layer_norm(x, self.weight, self.bias, self.eps, out_dtype)

    def extra_repr(self) -> str:
        return f"{self.channels}, eps={self.eps}, bias={self.bias is not None}"


class DropoutFunction(torch.autograd.Function):
    """``sequence.dropout``: the mask is made again from (seed, offset) in the
    backward pass, nothing is saved but an offset in device memory."""

    @staticmethod
    def forward(ctx, x, p, seed, offset, residual):
        ctx.key = (p, seed, offset)
        if isinstance(offset, torch.Tensor):
            ctx.key = (p, seed)
            ctx.save_for_backward(offset)
        ctx.residual = residual is not None
        return sequence.dropout(x, p, seed, offset, residual=residual)

    @staticmethod
    def backward(ctx, gy):
        gx = None
        if ctx.needs_input_grad[0]:
            # (differentiable again: the same linear map)
            gx = dropout(gy, *ctx.key, *ctx.saved_tensors)
        return gx, None, None, None, gy if ctx.residual else None


def dropout(x: torch.Tensor, p: float, seed: int, offset: Union[int, torch.Tensor] = 0,
            residual: Optional[torch.Tensor] = None) -> torch.Tensor:
    """residual + (kept ? x / (1 - p) : 0) with autograd; the mask is a
    function of (seed, offset, element index).  An offset in device memory
    must keep its value until the backward pass."""
    return DropoutFunction.apply(x.contiguous(), p, seed, offset,
                                 residual.contiguous() if residual is not None else None)


class DeltaRuleFunction(torch.autograd.Function):
    """``sequence.delta_rule`` and its gradients; only the inputs are saved.
    Differentiable once."""

    @staticmethod
    def forward(ctx, q, k, v, g, beta, s0, lengths, scale):
        ctx.set_materialize_grads(False)
        ctx.save_for_backward(q, k, v, g, beta, s0, lengths)
        ctx.scale = scale
        return sequence.delta_rule(q, k, v, g, beta, s0, lengths, scale)

    @staticmethod
    def backward(ctx, do, ds1):
        q, k, v, g, beta, s0, lengths = ctx.saved_tensors
        do = torch.zeros_like(v, memory_format=torch.contiguous_format) if do is None \
            else do.contiguous()
        ds1 = ds1.contiguous() if ds1 is not None else None
        return _gradients(functools.partial(sequence.delta_rule_bwd, scale=ctx.scale), do, ds1,
                          q, k, v, g, beta, s0, lengths) + (None, None)


def delta_rule(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, g: torch.Tensor,
               beta: torch.Tensor, s0: Optional[torch.Tensor] = None,
               lengths: Optional[torch.Tensor] = None, scale: Optional[float] = None
               ) -> Tuple[torch.Tensor, torch.Tensor]:
    """The gated delta rule over whole sequences with autograd: (o, s1).
    Shapes as ``sequence.delta_rule``; g, beta and the states are fp32."""
    return DeltaRuleFunction.apply(q, k, v, g, beta, s0, lengths, scale)


class MixerState(NamedTuple):
    """What a ``GatedDeltaMixer`` carries from token to token: the last
    kernel_size - 1 tokens of its convolution's input (b x taps x channels)
    and the states of the delta rule (b x value heads x dk x dv, fp32)."""

    taps: torch.Tensor
    states: torch.Tensor


_seeds = itertools.count()


class GatedDeltaMixer(torch.nn.Module):
    """A residual sequence layer on b x l x channels:

      h = layer_norm(x);  q, k, v = SiLU(causal depthwise convolution(h W_in))
      q, k normalised to length 1;  beta = sigmoid(h W_beta),
      g = -exp(a) softplus(h W_g + bias)
      o, state = delta_rule(q, k, v, g, beta, state)
      y = x + dropout(layer_norm(o) per head, times SiLU(h W_gate), times W_out)

    ``forward`` takes whole sequences (``lengths`` where they are unequal: y
    past a length is x) and returns (y, MixerState); ``step`` takes one token
    of each sequence and updates the state in place.

    Dropout is active in training; its masks are a function of ``seed`` (by
    default a number that no other layer of the process has) and of how many
    elements earlier calls covered.  That count is ``position``, a buffer on
    the device: it is saved with the parameters, and a captured step counts on
    with each replay.  A call that is recomputed in the backward pass
    (activation checkpointing) has to name its masks: ``forward(..., offset)``
    takes them there, from an int or an int64 value in device memory, and
    leaves the count alone; later calls are independent at offsets at least
    (numel + 3) // 4 apart."""

    def __init__(self, channels: int, heads: int, key_heads: Optional[int] = None,
                 key_dim: int = 128, value_dim: int = 128, kernel_size: int = 4,
                 p: float = 0.0, seed: Optional[int] = None, eps: float = 1e-5, device=None,
                 dtype=torch.float32):
        super().__init__()
        key_heads = heads if key_heads is None else key_heads
        if key_heads < 1 or heads % key_heads:
            raise ValueError("heads must be a multiple of key_heads")
        if not 1 <= key_dim <= 128:
            raise ValueError("key_dim must be 1..128")
        if kernel_size < 1:
            raise ValueError("kernel_size must be at least 1")
        if not 0.0 <= p <= 1.0:
            raise ValueError("p must be 0..1")
        self.heads, self.key_heads = int(heads), int(key_heads)
        self.key_dim, self.value_dim = int(key_dim), int(value_dim)
        self.kernel_size, self.p = int(kernel_size), float(p)
        self.seed = next(_seeds) if seed is None else int(seed)
        self.register_buffer("position", torch.zeros((), dtype=torch.int64, device=device))
        nk, nv = self.key_heads * self.key_dim, self.heads * self.value_dim
        self.mixed = 2 * nk + nv
        kw = dict(device=device, dtype=dtype)
        self.norm = LayerNorm(channels, eps, device=device)
        self.w_in = torch.nn.Linear(channels, self.mixed, bias=False, **kw)
        self.w_rate = torch.nn.Linear(channels, 2 * self.heads, bias=False, **kw)
        self.w_gate = torch.nn.Linear(channels, nv, bias=False, **kw)
        self.w_out = torch.nn.Linear(nv, channels, bias=False, **kw)
        self.conv = DepthwiseConv2d(self.mixed, (1, self.kernel_size),
                                    padding=(0, self.kernel_size - 1), layout="nhwc", **kw)
        self.out_norm = LayerNorm(self.value_dim, eps, device=device)
        f32 = dict(device=device, dtype=torch.float32)
        self.a = torch.nn.Parameter(torch.zeros(self.heads, **f32))
        self.g_bias = torch.nn.Parameter(torch.zeros(self.heads, **f32))

    @property
    def offset(self) -> int:
        """The value of ``position``: where the next call's masks begin."""
        return int(self.position)

    @offset.setter
    def offset(self, value: int) -> None:
        self.position.fill_(int(value))

    def _load_from_state_dict(self, state_dict, prefix, *args):
        # a state saved without the count leaves it as it is
        state_dict.setdefault(prefix + "position", self.position)
        super()._load_from_state_dict(state_dict, prefix, *args)

    def _rates(self, h):
        r = self.w_rate(h).float()
        g = -torch.exp(self.a) * F.softplus(r[..., :self.heads] + self.g_bias)
        return g, torch.sigmoid(r[..., self.heads:])

    def _heads(self, c):
        """q, k, v as heads, from the convolution's fp32 output."""
        dt = self.w_in.weight.dtype
        nk = self.key_heads * self.key_dim
        c = F.silu(c)
        qk = c[..., :2 * nk].unflatten(-1, (2 * self.key_heads, self.key_dim))
        qk = (qk * torch.rsqrt((qk * qk).sum(-1, keepdim=True) + 1e-6)).to(dt)
        v = c[..., 2 * nk:].unflatten(-1, (self.heads, self.value_dim)).to(dt)
        return qk[..., :self.key_heads, :], qk[..., self.key_heads:, :], v

    def _out(self, x, h, o, offset=None):
        y = self.w_out(self.out_norm(o).flatten(-2) * F.silu(self.w_gate(h)))
        y = y.to(x.dtype)
        if not self.training or self.p == 0.0:
            return x + y
        if offset is None:
            if torch._C._current_graph_task_id() != -1:
                raise RuntimeError("a call recomputed in the backward pass would take other "
                                   "dropout masks than the first one did: give both an offset")
            offset = self.position.clone()
            self.position += (y.numel() + 3) // 4
        return dropout(y, self.p, self.seed, offset, residual=x)

    def forward(self, x: torch.Tensor, state: Optional[MixerState] = None,
                lengths: Optional[torch.Tensor] = None,
                offset: Union[int, torch.Tensor, None] = None
                ) -> Tuple[torch.Tensor, MixerState]:
        b, n, _ = x.shape
        seen = x
        if lengths is not None:
            ends = lengths.clamp(0, n).long()
            live = (torch.arange(n, device=x.device) < ends[:, None])[..., None]
            # what stands past a length is not used, not even times a zero gradient
            seen = torch.where(live, x, 0.0)
        h = self.norm(seen, self.w_in.weight.dtype)
        m, taps = self.w_in(h), self.kernel_size - 1
        past = state.taps if state is not None else m.new_zeros(b, taps, self.mixed)
        m = torch.cat([past, m], 1)
        # of the outputs of a padded row, those that see no token past their own
        c = self.conv(m.unsqueeze(1))[:, 0, taps:taps + n]
        g, beta = self._rates(h)
        o, s1 = delta_rule(*self._heads(c), g, beta, state.states if state is not None else None,
                           lengths)
        y = self._out(x, h, o, offset)
        if lengths is None:
            # (a copy also where one sequence's part is contiguous as it is)
            return y, MixerState(m[:, n:].clone(memory_format=torch.contiguous_format), s1)
        at = ends[:, None] + torch.arange(taps, device=x.device)
        kept = m.gather(1, at[..., None].expand(-1, -1, self.mixed))
        return torch.where(live, y, x), MixerState(kept, s1)

    @torch.no_grad()
    def step(self, x: torch.Tensor, state: MixerState) -> torch.Tensor:
        """One token of each sequence (b x 1 x channels); ``state`` is updated
        in place."""
        if x.dim() != 3 or x.shape[1] != 1:
            raise ValueError(f"x must be b x 1 x channels, got {tuple(x.shape)}")
        h = self.norm(x, self.w_in.weight.dtype)
        m = torch.cat([state.taps, self.w_in(h)], 1)
        c = fwd(m.unsqueeze(1), self.conv.weight, 1, 0, algo=self.conv.algo)[:, 0]
        g, beta = self._rates(h)
        o, _ = sequence.delta_rule_step(*self._heads(c), g, beta, state.states,
                                        out_state=state.states)
        state.taps.copy_(m[:, 1:])
        return self._out(x, h, o)

    def extra_repr(self) -> str:
        return (f"heads={self.heads}, key_heads={self.key_heads}, key_dim={self.key_dim}, "
                f"value_dim={self.value_dim}, kernel_size={self.kernel_size}, p={self.p}")


def _typed(grad, like):
    """An fp32 gradient as the parameter's type has it."""
    return grad.to(like.dtype) if grad is not None else None


class CausalConvFunction(torch.autograd.Function):
    """``space.causal_conv`` and its gradients; only the inputs are saved.
    Differentiable once."""

    @staticmethod
    def forward(ctx, x, w, bias, s0, lengths, act):
        ctx.set_materialize_grads(False)
        ctx.save_for_backward(x, w, bias, s0, lengths)
        ctx.act = act
        return space.causal_conv(x, w, bias, s0, lengths, act)

    @staticmethod
    def backward(ctx, gy, gs):
        x, w, bias, s0, lengths = ctx.saved_tensors
        gy = torch.zeros_like(x, memory_format=torch.contiguous_format) if gy is None \
            else gy.contiguous()
        gs = gs.contiguous() if gs is not None else None
        dx, dw, dbias, ds0 = _gradients(functools.partial(space.causal_conv_bwd, act=ctx.act), gy,
                                        gs, x, w, bias, s0, lengths)
        return dx, _typed(dw, w), _typed(dbias, bias), ds0, None, None


def causal_conv(x: torch.Tensor, w: torch.Tensor, bias: Optional[torch.Tensor] = None,
                s0: Optional[torch.Tensor] = None, lengths: Optional[torch.Tensor] = None,
                act: str = "none") -> Tuple[torch.Tensor, torch.Tensor]:
    """Short causal depthwise convolution over tokens with autograd: (y, s1).
    Shapes as ``space.causal_conv``."""
    return CausalConvFunction.apply(x, w, bias, s0, lengths, act)


class SelectiveScanFunction(torch.autograd.Function):
    """``space.selective_scan`` and its gradients; only the inputs are saved.
    Differentiable once."""

    @staticmethod
    def forward(ctx, u, delta, A, B, C, D, z, delta_bias, s0, lengths, softplus):
        ctx.set_materialize_grads(False)
        ctx.save_for_backward(u, delta, A, B, C, D, z, delta_bias, s0, lengths)
        ctx.softplus = softplus
        return space.selective_scan(u, delta, A, B, C, D, z, delta_bias, s0, lengths, softplus)

    @staticmethod
    def backward(ctx, gy, gs):
        saved = ctx.saved_tensors
        gy = torch.zeros_like(saved[0], memory_format=torch.contiguous_format) if gy is None \
            else gy.contiguous()
        gs = gs.contiguous() if gs is not None else None
        return _gradients(functools.partial(space.selective_scan_bwd, softplus=ctx.softplus), gy,
                          gs, *saved) + (None, None)


def selective_scan(u: torch.Tensor, delta: torch.Tensor, A: torch.Tensor, B: torch.Tensor,
                   C: torch.Tensor, D: Optional[torch.Tensor] = None,
                   z: Optional[torch.Tensor] = None, delta_bias: Optional[torch.Tensor] = None,
                   s0: Optional[torch.Tensor] = None, lengths: Optional[torch.Tensor] = None,
                   softplus: bool = False) -> Tuple[torch.Tensor, torch.Tensor]:
    """The selective state space scan over whole sequences with autograd:
    (y, s1).  Shapes as ``space.selective_scan``; A, D, delta_bias and the
    states are fp32."""
    return SelectiveScanFunction.apply(u, delta, A, B, C, D, z, delta_bias, s0, lengths, softplus)


class ResidualNormFunction(torch.autograd.Function):
    """``space.residual_norm`` and its gradients; the inputs and a value a row
    of each norm are saved.  Differentiable once."""

    @staticmethod
    def forward(ctx, x, y, gate, scale, w_post, w_pre, eps, post, pre, act):
        ctx.set_materialize_grads(False)
        r, h, q1, q2 = space.residual_norm(x, y, gate, scale, w_post, w_pre, eps, post, pre, act)
        ctx.save_for_backward(x, y, q1, q2, gate, scale, w_post, w_pre)
        ctx.how = dict(post=post, pre=pre, act=act)
        return r, h

    @staticmethod
    def backward(ctx, gr, gh):
        x, y, q1, q2, gate, scale, w_post, w_pre = ctx.saved_tensors
        if gr is None and gh is None:
            return (None,) * 10
        gr = gr.contiguous() if gr is not None else None
        gh = gh.contiguous() if gh is not None else None
        dx, dy, dgate, *sums = _gradients(functools.partial(space.residual_norm_bwd, **ctx.how),
                                          gr, gh, x, y, q1, q2, gate, scale, w_post, w_pre)
        return (dx, dy, dgate, *map(_typed, sums, (scale, w_post, w_pre)), None, None, None, None)


def _rows(t):
    """A matrix with a row stride as it is, other views made contiguous."""
    if t is None or (t.dim() == 2 and t.stride(1) == 1 and t.stride(0) >= t.shape[1]):
        return t
    return t.contiguous()


def residual_norm(x: Optional[torch.Tensor], y: torch.Tensor,
                  gate: Optional[torch.Tensor] = None, scale: Optional[torch.Tensor] = None,
                  w_post: Optional[torch.Tensor] = None, w_pre: Optional[torch.Tensor] = None,
                  eps: float = 1e-5, post: bool = True, pre: bool = True, act: str = "none"
                  ) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """r = x + scale act(gate) norm(y) w_post and h = norm(r) w_pre over the
    last axis with autograd: (r, h), as ``space.residual_norm``."""
    return ResidualNormFunction.apply(_rows(x), _rows(y), _rows(gate), scale, w_post, w_pre, eps,
                                      post, pre, act)


def rms_norm(y: torch.Tensor, w: Optional[torch.Tensor] = None,
             gate: Optional[torch.Tensor] = None, eps: float = 1e-5,
             act: str = "silu") -> torch.Tensor:
    """y / sqrt(mean(y^2) + eps) w over the last axis, times act(gate) where a
    gate is given, with autograd."""
    return residual_norm(None, y, gate, None, w, None, eps, pre=False, act=act)[0]


class ScanState(NamedTuple):
    """What a ``SelectiveScanMixer`` carries from token to token: the last
    kernel_size - 1 inputs of its convolution (b x taps x inner) and the
    states of the scan (b x inner x states, fp32)."""

    taps: torch.Tensor
    states: torch.Tensor


class SelectiveScanMixer(torch.nn.Module):
    """A selective state space mixer on b x l x channels:

      x, z = h W_in;  u = SiLU(causal depthwise convolution(x))
      low, B, C = u W_x;  delta = low W_dt
      y = selective_scan(u, softplus(delta + bias), -exp(a), B, C, D, gate z) W_out

    ``forward`` takes whole sequences (``lengths`` where they are unequal: y
    past a length is 0) and returns (y, ScanState); ``step`` takes one or a
    few tokens of each sequence and updates the state in place."""

    def __init__(self, channels: int, inner: Optional[int] = None, states: int = 16,
                 kernel_size: int = 4, rank: Optional[int] = None, groups: int = 1, device=None,
                 dtype=torch.float32):
        super().__init__()
        self.inner = int(2 * channels if inner is None else inner)
        self.states, self.kernel_size, self.groups = int(states), int(kernel_size), int(groups)
        self.rank = max(1, -(-int(channels) // 16)) if rank is None else int(rank)
        if not 1 <= self.states <= 256:
            raise ValueError("states must be 1..256")
        if not 1 <= self.kernel_size <= 8:
            raise ValueError("kernel_size must be 1..8")
        if self.groups < 1 or self.inner % self.groups:
            raise ValueError("inner must be a multiple of groups")
        if self.rank < 1:
            raise ValueError("rank must be at least 1")
        kw = dict(device=device, dtype=dtype)
        self.w_in = torch.nn.Linear(channels, 2 * self.inner, bias=False, **kw)
        self.w_x = torch.nn.Linear(self.inner, self.rank + 2 * self.groups * self.states,
                                   bias=False, **kw)
        self.w_dt = torch.nn.Linear(self.rank, self.inner, bias=False, **kw)
        self.w_out = torch.nn.Linear(self.inner, channels, bias=False, **kw)
        self.conv_weight = torch.nn.Parameter(torch.empty(self.kernel_size, self.inner, **kw))
        self.conv_bias = torch.nn.Parameter(torch.zeros(self.inner, **kw))
        f32 = dict(device=device, dtype=torch.float32)
        self.a = torch.nn.Parameter(
            torch.arange(1, self.states + 1, **f32).log().repeat(self.inner, 1))
        self.D = torch.nn.Parameter(torch.ones(self.inner, **f32))
        # steps from 0.001 to 0.1, even in their logarithm, where delta is 0
        step = torch.exp(torch.rand(self.inner, **f32) * math.log(100.0) + math.log(1e-3))
        self.delta_bias = torch.nn.Parameter(step + torch.log(-torch.expm1(-step)))
        bound = 1.0 / math.sqrt(self.kernel_size)
        with torch.no_grad():
            self.conv_weight.uniform_(-bound, bound)

    def _operands(self, u):
        """delta, A, B, C of the convolution's output."""
        g, n = self.groups, self.states
        mixed = self.w_x(u)
        delta = self.w_dt(mixed[..., :self.rank])
        B = mixed[..., self.rank:self.rank + g * n].unflatten(-1, (g, n))
        C = mixed[..., self.rank + g * n:].unflatten(-1, (g, n))
        return delta, -torch.exp(self.a.float()), B, C

    def _vectors(self):
        """D and the steps' bias, fp32 also in a module converted as a whole."""
        return self.D.float(), self.delta_bias.float()

    def forward(self, h: torch.Tensor, state: Optional[ScanState] = None,
                lengths: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, ScanState]:
        if lengths is not None:
            live = torch.arange(h.shape[1], device=h.device) < lengths[:, None]
            # what stands past a length is not used, not even times a zero gradient
            h = torch.where(live[..., None], h, 0.0)
        xz = self.w_in(h)
        taps, states = state if state is not None else (None, None)
        u, taps = causal_conv(xz[..., :self.inner], self.conv_weight, self.conv_bias, taps,
                              lengths, "silu")
        D, bias = self._vectors()
        y, states = selective_scan(u, *self._operands(u), D, xz[..., self.inner:], bias, states,
                                   lengths, softplus=True)
        return self.w_out(y), ScanState(taps, states)

    @torch.no_grad()
    def step(self, h: torch.Tensor, state: ScanState) -> torch.Tensor:
        """One or a few tokens of each sequence (b x l x channels); ``state``
        is updated in place."""
        xz = self.w_in(h)
        u, _ = space.causal_conv_step(xz[..., :self.inner], self.conv_weight, self.conv_bias,
                                      state.taps, act="silu", out_state=state.taps)
        D, bias = self._vectors()
        y, _ = space.selective_scan_step(u, *self._operands(u), D, xz[..., self.inner:], bias,
                                         state.states, softplus=True, out_state=state.states)
        return self.w_out(y)

    def extra_repr(self) -> str:
        return (f"inner={self.inner}, states={self.states}, kernel_size={self.kernel_size}, "
                f"rank={self.rank}, groups={self.groups}")


class SelectiveScanLayers(torch.nn.Module):
    """Selective state space mixers on a residual stream of b x l x channels,
    with RMS norms before and behind each:

      h = norm(x);  for each layer:  y = mixer(h)
      x = x + scale norm(y) w_post,  h = norm(x) w_pre of the next layer

    the last two in one pass (``residual_norm``).  ``forward`` returns (the
    last h, 0 past a length, and the states of each layer); ``step`` takes one
    or a few tokens and updates the states in place.  The stream keeps x's type, fp32 or the
    mixers'."""

    def __init__(self, channels: int, layers: int, eps: float = 1e-5, scale: float = 1.0,
                 device=None, dtype=torch.float32, **mixer):
        super().__init__()
        self.eps = float(eps)
        self.mixers = torch.nn.ModuleList(
            SelectiveScanMixer(channels, device=device, dtype=dtype, **mixer)
            for _ in range(layers))
        new = lambda k, v: torch.nn.Parameter(  # noqa: E731
            torch.full((k, channels), v, device=device, dtype=torch.float32))
        self.w_pre, self.w_post = new(layers + 1, 1.0), new(layers, 1.0)
        self.scale = new(layers, float(scale))

    def _run(self, x, call):
        dt = self.mixers[0].w_in.weight.dtype if len(self.mixers) else x.dtype
        # unbind: the gradients of the rows are joined by one operation
        pre, post, scale = self.w_pre.unbind(), self.w_post.unbind(), self.scale.unbind()
        h = rms_norm(x, pre[0], eps=self.eps).to(dt)
        for i in range(len(self.mixers)):
            x, h = residual_norm(x, call(i, h), None, scale[i], post[i], pre[i + 1], self.eps)
        return h

    def forward(self, x: torch.Tensor, state: Optional[List[ScanState]] = None,
                lengths: Optional[torch.Tensor] = None
                ) -> Tuple[torch.Tensor, List[ScanState]]:
        after: List[ScanState] = []
        if lengths is not None:
            live = torch.arange(x.shape[1], device=x.device) < lengths[:, None]
            # (the norms' gradients see no row past a length)
            x = torch.where(live[..., None], x, 0.0)

        def call(i, h):
            y, s = self.mixers[i](h, state[i] if state is not None else None, lengths)
            after.append(s)
            return y

        return self._run(x, call), after

    @torch.no_grad()
    def step(self, x: torch.Tensor, state: List[ScanState]) -> torch.Tensor:
        return self._run(x, lambda i, h: self.mixers[i].step(h, state[i]))
