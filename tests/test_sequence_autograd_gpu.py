"""The sequence operators under autograd's rules: no buffer is changed behind
a graph that saved it, no second derivative vanishes silently."""

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import depthwise_convolution_dwc_amd.nn as dnn  # noqa: E402
from gpu_helpers import dwc, sync  # noqa: E402
from test_mixer_gpu import mixer  # noqa: E402
from test_sequence_gpu import F32, delta_inputs, randn  # noqa: E402


def test_state_updated_before_backward_raises():
    a = [t.clone().requires_grad_() for t in delta_inputs(5, 2, 70, 1, 2, 16, 8, F32)]
    token = [t[:, :1].detach() for t in a[:5]]
    state = a[5].detach().clone()
    o, s1 = dnn.delta_rule(*a[:5], state)
    dwc.delta_rule_step(*token, state, out_state=state)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        o.sum().backward()
    m = mixer()
    x = randn(6, 2, 20, 64)
    with torch.no_grad():
        state = m(x)[1]
    y, _ = m(x, state)
    m.step(x[:, :1], state)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.sum().backward()


@pytest.mark.parametrize("which", ["layer norm", "dropout"])
def test_output_written_before_backward_raises(which):
    x, kept = randn(7, 6, 40), randn(8, 6, 40)
    w = torch.ones(6, 40, device="cuda", requires_grad=True)
    y = (w * kept).sum()
    if which == "layer norm":
        dwc.layer_norm(x, out=kept)
    else:
        dwc.dropout(x, 0.5, 1, out=kept)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward()


def test_outputs_given_without_autograd():
    """Buffers that have no version counter are written all the same."""
    with torch.inference_mode():
        x = randn(9, 6, 40)
        out = torch.empty_like(x)
        assert dwc.layer_norm(x, out=out)[0] is out
        sync()
        assert torch.equal(out, dwc.layer_norm(x)[0])
        a = delta_inputs(10, 2, 1, 1, 2, 16, 8, F32)
        s = a[5].clone()
        o, s1 = dwc.delta_rule_step(*a[:5], s, out_state=s)
        assert s1 is s and torch.equal(s, dwc.delta_rule_step(*a)[1])


def second(out, leaf):
    """The gradient of a penalty on a gradient."""
    g = torch.autograd.grad(out.square().sum(), leaf, create_graph=True)[0]
    return torch.autograd.grad(g.square().sum() + leaf.sum(), leaf)[0]


def test_second_derivatives():
    x, w = randn(1, 6, 40).requires_grad_(), randn(2, 40)
    with pytest.raises(RuntimeError, match="differentiable once"):
        second(dnn.layer_norm(x, w), x)
    a = [t.clone().requires_grad_() for t in delta_inputs(4, 1, 5, 1, 1, 8, 8, F32)]
    with pytest.raises(RuntimeError, match="differentiable once"):
        second(dnn.delta_rule(*a)[0], a[2])
    # y = 2 x where kept: the gradient is 8 x there, its penalty's 128 x + 1
    x, r = randn(3, 50).requires_grad_(), randn(5, 50)
    kept = dwc.dropout(torch.ones_like(x), 0.5, 7).bool()
    want = torch.where(kept, 128 * x.detach() + 1, 1.0)
    assert torch.equal(second(dnn.dropout(x, 0.5, 7), x), want)
    at = torch.zeros((), dtype=torch.int64, device="cuda")
    assert torch.equal(second(dnn.dropout(x, 0.5, 7, at), x), want)
    y = dnn.dropout(x, 0.5, 7, residual=r)
    g = torch.autograd.grad(y, x, torch.ones_like(y), create_graph=True)[0]
    assert torch.equal(g, 2.0 * kept)
