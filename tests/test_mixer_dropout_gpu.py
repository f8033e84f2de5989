"""The masks of ``GatedDeltaMixer``: other ones for each call, layer and
replay, the same ones for a recomputed call and after a restart."""

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

from torch.utils.checkpoint import checkpoint  # noqa: E402

import depthwise_convolution_dwc_amd.nn as dnn  # noqa: E402
from gpu_helpers import dwc, log, sync  # noqa: E402
from test_mixer_gpu import mixer  # noqa: E402
from test_sequence_gpu import BF16, F16, F32, randn  # noqa: E402


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("n", [1, 7, 4096, 65537])
def test_position_in_device_memory(dtype, n):
    """An offset that the kernel reads gives the bits of one given by value,
    also where their sum passes 64 bits."""
    log(f"case position {dtype} {n}")
    x, r = randn(n, n, dtype=dtype), randn(n + 1, n, dtype=dtype)
    for at in (0, 5, (1 << 40) + 3, (1 << 64) - 2):
        p = torch.tensor(at - (1 << 64) if at >> 63 else at, device="cuda")
        for res in (None, r):
            assert torch.equal(dwc.dropout(x, 0.4, 11, p, residual=res),
                               dwc.dropout(x, 0.4, 11, at, residual=res))
    z = x.clone().requires_grad_()
    dnn.dropout(z, 0.4, 11, p).float().sum().backward()
    assert torch.equal(z.grad, dwc.dropout(torch.ones_like(x), 0.4, 11, at))


def test_position_refused():
    x = randn(1, 8)
    for bad in (torch.zeros(2, dtype=torch.int64, device="cuda"), torch.tensor(3)):
        with pytest.raises(ValueError):
            dwc.dropout(x, 0.5, 1, bad)
    with pytest.raises(TypeError):
        dwc.dropout(x, 0.5, 1, torch.zeros((), device="cuda"))


def grads(m, run, x, gy):
    z = x.clone().requires_grad_()
    y = run(z)
    return (y.detach(),) + torch.autograd.grad(y, (z,) + tuple(m.parameters()), gy,
                                               allow_unused=True)


@pytest.mark.parametrize("reentrant", [False, True])
def test_recomputed_call(reentrant):
    """A call that is made again in the backward pass has to name its masks."""
    m = mixer(p=0.3, seed=2).train()
    x, gy = randn(2, 2, 30, 64), randn(3, 2, 30, 64)
    z = x.clone().requires_grad_()
    y, _ = checkpoint(m, z, use_reentrant=reentrant)
    with pytest.raises(RuntimeError, match="offset"):
        (y * gy).sum().backward()
    del y
    at = m.offset
    want = grads(m, lambda z: m(z, offset=77)[0], x, gy)
    z = x.clone().requires_grad_()
    y, _ = checkpoint(m, z, None, None, 77, use_reentrant=reentrant)
    (y * gy).sum().backward()
    assert torch.equal(y.detach(), want[0]) and torch.equal(z.grad, want[1])
    for p, w in zip(m.parameters(), want[2:]):
        assert torch.equal(p.grad, w)
    assert m.offset == at  # a call that names its masks leaves the count alone


def test_layers_and_restarts():
    def layer(**kw):
        torch.manual_seed(4)
        return dnn.GatedDeltaMixer(64, heads=4, key_heads=2, key_dim=16, value_dim=24, p=0.5,
                                   device="cuda", **kw)

    a, b, c, d = layer(), layer(), layer(seed=9), layer(seed=9)
    x = randn(4, 2, 30, 64)
    y = [m(x)[0] for m in (a, b, c, d)]
    assert not torch.equal(y[0], y[1])  # two layers of one stack
    assert torch.equal(y[2], y[3])
    c(x)
    saved = c.state_dict()
    d.load_state_dict(saved)
    assert c.offset == d.offset == 2 * (x.numel() // 4)
    assert torch.equal(c(x)[0], d(x)[0])
    # a state without the count, as saved before there was one
    old = {k: v for k, v in saved.items() if k in dict(c.named_parameters())}
    e = layer(seed=9)
    e.load_state_dict(old)
    assert e.offset == 0


def test_captured_training_step():
    """Each replay has masks of its own, and the gradients belong to them."""
    m = mixer(p=0.5, seed=3).train()
    x, gy = randn(5, 2, 30, 64), randn(6, 2, 30, 64)
    z = x.clone().requires_grad_()
    leaves = (z,) + tuple(m.parameters())

    def step():
        y = m(z)[0]
        return (y,) + torch.autograd.grad(y, leaves, gy)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(2):
            step()
    side.synchronize()
    m.offset = 0
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        outs = step()
    assert m.offset == 0  # captured, not run
    seen = []
    for i in range(4):
        graph.replay()
        sync()
        assert m.offset == (i + 1) * (x.numel() // 4)
        want = grads(m, lambda t: m(t, offset=i * (x.numel() // 4))[0], x, gy)
        for s, t in zip(outs, want):
            assert torch.equal(s.detach(), t), i
        seen.append(outs[0].detach().clone())
        torch.randn(1000, 1000, device="cuda").sum().item()
    assert len({tuple(t.flatten().tolist()) for t in seen}) == 4
