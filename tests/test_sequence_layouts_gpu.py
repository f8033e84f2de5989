"""The sequence operators on operands laid out in other ways than the layer
makes them: heads before tokens, broadcast axes, strided gradients, many
tokens, and offsets that pass 32 bits.  References and bounds are those of
test_delta_gpu.py and test_sequence_gpu.py."""

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import test_delta_gpu as delta  # noqa: E402
from gpu_helpers import dwc, log, sync  # noqa: E402
from test_delta_gpu import F, TOL  # noqa: E402
from test_sequence_gpu import (BF16, F16, F32, delta_inputs, delta_reference, half,  # noqa: E402
                               randn, rel)


def heads_first(t):
    """The same values with heads before tokens in memory."""
    return t.transpose(1, 2).contiguous().transpose(1, 2)


def tokens_first(t):
    return t.transpose(0, 1).contiguous().transpose(0, 1)


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("order", [heads_first, tokens_first])
@pytest.mark.parametrize("shape", [(2, 130, 2, 4, 64, 64), (3, 70, 2, 2, 100, 75),
                                   (9, 66, 8, 16, 128, 48)])
def test_delta_operand_orders(dtype, order, shape):
    log(f"case order {dtype} {order.__name__} {shape}")
    a = delta_inputs(sum(shape), *shape, dtype)
    views = [order(t) for t in a[:5]] + [a[5]]
    o, s1, grads = delta.check(views)
    b, n, hk, hv, dk, dv = shape
    for pad in (0, 3):  # a gradient in the same order, and with gaps between its heads
        dout = order(randn(2, b, n, hv, dv + pad, dtype=dtype))[..., :dv]
        ds1 = randn(3, b, hv, dk, dv, scale=0.1)
        got = dwc.delta_rule_bwd(dout, ds1, *views)
        same = dwc.delta_rule_bwd(dout.contiguous(), ds1, *views)
        sync()
        for x, y in zip(got, same):
            assert torch.equal(x, y)
    head = [t[:, :2] for t in views[:5]] + [a[5]]
    o, s1 = dwc.delta_rule_step(*head)
    wo, ws = delta_reference(*head)
    assert rel(s1, ws) < F and rel(o, wo) < half(dtype) + F


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_delta_broadcast_operands(dtype):
    """Axes of stride 0: one decay for all heads, one q for all sequences."""
    log(f"case broadcast {dtype}")
    q, k, v, g, beta, s0 = delta_inputs(4, 3, 100, 2, 4, 48, 40, dtype)
    a = [q[:1].expand(3, 100, 2, 48), k[:, :, :1].expand(3, 100, 2, 48), v,
         g[:, :, :1].expand(3, 100, 4), beta[:, :1].expand(3, 100, 4), s0]
    delta.check(a)
    lengths = torch.tensor([100, 0, 65], dtype=torch.int32, device="cuda")
    delta.check(a, lengths)
    dout = randn(5, 1, 1, 1, 40, dtype=dtype).expand(3, 100, 4, 40)
    for x, y in zip(dwc.delta_rule_bwd(dout, None, *a),
                    dwc.delta_rule_bwd(dout.contiguous(), None, *a)):
        assert torch.equal(x, y)
    o, s1 = dwc.delta_rule_step(*(t[:, :2] for t in a[:5]), s0)
    wo, ws = delta_reference(*(t[:, :2] for t in a[:5]), s0)
    assert rel(s1, ws) < F and rel(o, wo) < half(dtype) + F


@pytest.mark.parametrize("dtype,shape", [(F32, (1, 2100, 1, 2, 64, 64)),
                                         (BF16, (2, 1500, 2, 2, 128, 64)),
                                         (F16, (1, 3001, 1, 1, 40, 130))])
def test_delta_many_tokens(dtype, shape):
    log(f"case many tokens {dtype} {shape}")
    delta.check(delta_inputs(sum(shape), *shape, dtype))


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_delta_offsets_past_32_bits(dtype):
    """Two sequences, 2^32 and more elements apart."""
    log(f"case far {dtype}")
    a = list(delta_inputs(6, 2, 70, 1, 2, 64, 40, dtype))
    b, n, hv, dv = a[2].shape
    dout, ds1 = randn(7, b, n, hv, dv, dtype=dtype), randn(8, b, hv, 64, dv, scale=0.1)
    want = dwc.delta_rule(*a) + dwc.delta_rule_bwd(dout, ds1, *a)
    token = dwc.delta_rule_step(*(t[:, :1] for t in a[:5]), a[5])
    far = (1 << 32) + 8
    store = torch.empty(far + (1 << 20), dtype=dtype, device="cuda")

    def apart(t, at):
        s = t.contiguous().stride()
        view = store.as_strided(t.shape, (far,) + s[1:], at)
        return view.copy_(t)

    at, views = 0, []
    for t in a[:3] + [dout]:
        views.append(apart(t, at))
        at += t[0].numel() + 8
    got = dwc.delta_rule(*views[:3], *a[3:]) + dwc.delta_rule_bwd(views[3], ds1, *views[:3], *a[3:])
    sync()
    for x, y in zip(got, want):
        assert rel(x, y.double()) <= 2 * TOL[x.dtype]
    for x, y in zip(dwc.delta_rule_step(*(t[:, :1] for t in views[:3]),
                                        *(t[:, :1] for t in a[3:5]), a[5]), token):
        assert rel(x, y.double()) <= 2 * (half(x.dtype) + F)


def test_norm_and_dropout_offsets_past_32_bits():
    log("case far norm")
    far = (1 << 31) + 64
    store = torch.empty(2 * far + 4096, dtype=BF16, device="cuda")
    x = store.as_strided((3, 512), (far, 1)).copy_(randn(9, 3, 512, dtype=BF16))
    dy = store.as_strided((3, 512), (far, 1), 1024).copy_(randn(10, 3, 512, dtype=BF16))
    y, mean, rstd = dwc.layer_norm(x)
    for s, t in zip((y, mean, rstd) + dwc.layer_norm_bwd(dy, x, mean, rstd),
                    dwc.layer_norm(x.contiguous())
                    + dwc.layer_norm_bwd(dy.contiguous(), x.contiguous(), mean, rstd)):
        assert torch.equal(s, t)
    del x, dy
    n = (1 << 32) + 1003
    x = store[:n].normal_()
    y = dwc.dropout(x, 0.25, 5, 7)
    for at in (0, (1 << 31) - 2048, (1 << 32) - 1024):
        assert torch.equal(y[at:at + 2027], dwc.dropout(x[at:at + 2027], 0.25, 5, 7 + at // 4))
