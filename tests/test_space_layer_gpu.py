"""The causal convolution, the selective scan and the residual norm together,
as ``SelectiveScanMixer`` and ``SelectiveScanLayers`` run them: against a
plain 64-bit model, in pieces, captured into graphs, on other streams and
under autograd."""

import copy

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

from depthwise_convolution_dwc_amd.nn import (ScanState, SelectiveScanLayers,  # noqa: E402
                                              SelectiveScanMixer, causal_conv, residual_norm,
                                              rms_norm, selective_scan)
from gpu_helpers import dwc, log, sync  # noqa: E402
from test_sequence_gpu import BF16, F16, F32, randn  # noqa: E402
from test_scan_gpu import inputs  # noqa: E402


def plain_norm(v, w, eps):
    return v / torch.sqrt((v * v).mean(-1, keepdim=True) + eps) * w


def plain_mixer(m, p, h, lens):
    """``SelectiveScanMixer`` in 64 bits with the parameters p, one sequence at
    a time: (y, taps, states)."""
    ys, taps, states = [], [], []
    for i in range(h.shape[0]):
        n = lens[i] if lens is not None else h.shape[1]
        xz = h[i, :n] @ p["w_in.weight"].t()
        x, z = xz[:, :m.inner], xz[:, m.inner:]
        full = torch.cat([x.new_zeros(m.kernel_size - 1, m.inner), x])
        u = p["conv_bias"] + sum(p["conv_weight"][j] * full[j:j + n] for j in range(m.kernel_size))
        u = u * torch.sigmoid(u)
        mixed = u @ p["w_x.weight"].t()
        dt = torch.nn.functional.softplus(mixed[:, :m.rank] @ p["w_dt.weight"].t()
                                          + p["delta_bias"], threshold=100)
        each = lambda t: t.unflatten(-1, (m.groups, -1)).repeat_interleave(  # noqa: E731
            m.inner // m.groups, -2)
        B = each(mixed[:, m.rank:m.rank + m.groups * m.states])
        C = each(mixed[:, m.rank + m.groups * m.states:])
        s, o = x.new_zeros(m.inner, m.states), []
        for t in range(n):
            s = torch.exp(-dt[t, :, None] * torch.exp(p["a"])) * s + (dt[t] * u[t])[:, None] * B[t]
            o.append((s * C[t]).sum(-1) + p["D"] * u[t])
        o = torch.stack(o) if o else x
        y = (o * z * torch.sigmoid(z)) @ p["w_out.weight"].t()
        ys.append(torch.cat([y, y.new_zeros(h.shape[1] - n, y.shape[1])]))
        taps.append(full[n:])
        states.append(s)
    return torch.stack(ys), torch.stack(taps), torch.stack(states)


def plain_layers(m, p, x, lens):
    states = []
    if lens is not None:
        ends = torch.tensor(lens, device=x.device)
        x = torch.where((torch.arange(x.shape[1], device=x.device) < ends[:, None])[..., None],
                        x, 0.0)
    h = plain_norm(x, p["w_pre"][0], m.eps)
    for i, mixer in enumerate(m.mixers):
        sub = {k[len(f"mixers.{i}."):]: v for k, v in p.items() if k.startswith(f"mixers.{i}.")}
        y, taps, s = plain_mixer(mixer, sub, h, lens)
        states.append((taps, s))
        x = x + p["scale"][i] * plain_norm(y, p["w_post"][i], m.eps)
        h = plain_norm(x, p["w_pre"][i + 1], m.eps)
    return h, states


def near(got, want, tol, what):
    err = ((got.double() - want).norm() / (want.norm() + 1e-30)).item()
    log(f"{what}: {err:.2e} of {tol:.0e}")
    assert err <= tol, what


@pytest.mark.parametrize("lens", [None, [21, 0, 9]])
@pytest.mark.parametrize("groups,states", [(1, 16), (2, 5)])
def test_layers_and_gradients(lens, groups, states):
    """fp32 against 64 bits.  A fp32 product of K values is off by at most
    K u of its magnitudes and chains of ten such follow each other: 1e-4 in
    norm leaves room for magnitudes ten times the values."""
    log(f"case layers {lens} {groups} {states}")
    torch.manual_seed(0)
    m = SelectiveScanLayers(24, 2, scale=0.5, device="cuda", inner=36, states=states,
                            groups=groups, rank=3)
    x = randn(1, 3, 21, 24).requires_grad_()
    lengths = torch.tensor(lens, dtype=torch.int32, device="cuda") if lens else None
    p = {k: v.detach().double().requires_grad_() for k, v in m.named_parameters()}
    xd = x.detach().double().requires_grad_()
    want, after = plain_layers(m, p, xd, lens)
    gy = randn(2, 3, 21, 24)
    if lens:
        live = (torch.arange(21, device="cuda") < lengths[:, None])[..., None]
        want = torch.where(live, want, 0.0)
        with torch.no_grad():
            x.masked_fill_(~live, float("nan"))  # not used
    got, state = m(x, lengths=lengths)
    (got * gy).sum().backward()
    (want * gy.double()).sum().backward()
    sync()
    near(got, want.detach(), 1e-4, "h")
    for s, (taps, st) in zip(state, after):
        near(s.taps, taps.detach(), 1e-4, "taps")
        near(s.states, st.detach(), 1e-4, "states")
    near(x.grad, xd.grad, 1e-4, "dx")
    for k, v in m.named_parameters():
        near(v.grad, p[k].grad, 1e-4, k)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_prompt_then_tokens(dtype):
    """A prompt and single tokens behind it give what the whole gives.  The
    two differ where sums run in another order, 16-bit values by a rounding
    of each of the five operands in a row, 2^-8 each."""
    torch.manual_seed(1)
    m = SelectiveScanMixer(32, states=16, device="cuda", dtype=dtype)
    x = randn(3, 2, 19, 32, dtype=dtype)
    with torch.no_grad():
        whole, end = m(x)
        y, state = m(x[:, :12])
        out = [y] + [m.step(x[:, 12:14], state)] + [m.step(x[:, t:t + 1], state) for t in range(14, 19)]
    tol = 1e-5 if dtype == F32 else 5 * 2.0 ** -8
    near(torch.cat(out, 1), whole.double(), tol, "y")
    near(state.states, end.states.double(), tol, "states")
    near(state.taps, end.taps.double(), tol, "taps")


def test_unequal_prompts_then_tokens():
    torch.manual_seed(2)
    m = SelectiveScanLayers(16, 2, device="cuda", states=4, kernel_size=3)
    x = randn(4, 3, 11, 16)
    lens = [11, 5, 1]
    with torch.no_grad():
        h, state = m(x, lengths=torch.tensor(lens, dtype=torch.int32, device="cuda"))
        tok = randn(5, 3, 1, 16)
        got = m.step(tok, state)
        for i, n in enumerate(lens):
            alone, _ = m(torch.cat([x[i:i + 1, :n], tok[i:i + 1]], 1))
            near(h[i:i + 1, :n], alone[:, :n].double(), 1e-5, "prompt")
            near(got[i:i + 1], alone[:, n:].double(), 1e-5, "token")
            assert (h[i, n:] == 0).all()


def test_readme_example_runs():
    m = SelectiveScanLayers(256, layers=2, device="cuda", dtype=BF16)
    x = randn(1, 2, 70, 256, dtype=BF16).requires_grad_()
    h, state = m(x)
    h.float().sum().backward()
    assert h.dtype == BF16 and torch.isfinite(h).all()
    for k, v in m.named_parameters():
        assert v.grad is not None and torch.isfinite(v.grad).all() and v.grad.dtype == v.dtype, k
    h, state = m(x)
    assert m.step(x[:, -1:], [ScanState(*(t.detach() for t in s)) for s in state]).shape == (2, 1, 256)
    # an fp32 residual stream beside bf16 mixers
    h, _ = m(x.detach().float())
    assert h.dtype == BF16


def test_captured_training_step():
    """Replays of a captured step give the eager step's gradients, with eager
    work and synchronisations between them."""
    torch.manual_seed(3)
    m = SelectiveScanLayers(64, 2, device="cuda", dtype=BF16)
    ref = copy.deepcopy(m)
    x = torch.zeros(2, 150, 64, device="cuda", dtype=BF16)
    lengths = torch.tensor([150, 90], dtype=torch.int32, device="cuda")

    def step(m, x):
        h, _ = m(x, lengths=lengths)
        return torch.autograd.grad(h.float().square().sum(), list(m.parameters()))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(2):
            step(m, x)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(m, x)
    for i in range(4):
        x.copy_(randn(20 + i, 2, 150, 64, dtype=BF16))
        graph.replay()
        sync()
        want = step(ref, x.clone())
        sync()
        for (k, _), s, t in zip(m.named_parameters(), out, want):
            # the projections' products may run in another order
            near(s, t.double(), 1e-2, k)


def test_captured_operators_repeat_their_bits():
    """Two captured graphs with workspaces of their own, replayed in turn."""
    a = inputs(1, 2, 200, 96, 16, 1, BF16)
    w = randn(2, 4, 96, dtype=BF16)
    state, taps = a[8].clone(), randn(3, 2, 3, 96, dtype=BF16)
    one = [t[:, :1].contiguous() if t is not None and i in (0, 1, 3, 4, 6) else t
           for i, t in enumerate(a)]

    def work():
        y, s1 = dwc.selective_scan(*a, softplus=True)
        g = dwc.selective_scan_bwd(y, s1, *a, softplus=True)
        c = dwc.causal_conv(a[0], w, act="silu")
        cg = dwc.causal_conv_bwd(a[1], None, a[0], w, act="silu")
        r = dwc.residual_norm(a[0], a[1], gate=a[1], act="silu")
        n = dwc.residual_norm_bwd(a[0], a[1], a[0], a[1], r[2], r[3], gate=a[1], act="silu")
        t, _ = dwc.selective_scan_step(*one[:8], state, softplus=True, out_state=state)
        q, _ = dwc.causal_conv_step(one[0], w, None, taps, out_state=taps)
        return [v for v in (y, s1, *g, *c, *cg, *r, *n, t, q) if v is not None]

    begin = [state.clone(), taps.clone()]

    def reset():
        state.copy_(begin[0])
        taps.copy_(begin[1])

    work()
    graphs = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        sync()
        with torch.cuda.graph(graph):
            out = work()
        graphs.append((graph, out))
    for i in range(5):
        a[0].copy_(randn(30 + i, 2, 200, 96, dtype=BF16))
        one[0].copy_(a[0][:, :1])
        reset()
        want = [t.clone() for t in work()] + [state.clone(), taps.clone()]
        for graph, out in graphs:
            reset()
            sync()
            graph.replay()
            sync()
            for s, t in zip(out + [state, taps], want):
                assert torch.equal(s, t)


def calls():
    a = inputs(1, 2, 300, 256, 16, 1, BF16)
    w, taps = randn(2, 4, 256, dtype=BF16), randn(3, 2, 3, 256, dtype=BF16)
    r, h, q1, q2 = dwc.residual_norm(a[0], a[1])
    return {"causal_conv": lambda s: dwc.causal_conv(a[0], w, stream=s),
            "causal_conv_step": lambda s: dwc.causal_conv_step(a[0], w, None, taps, stream=s),
            "causal_conv_bwd": lambda s: dwc.causal_conv_bwd(a[1], None, a[0], w, stream=s),
            "selective_scan": lambda s: dwc.selective_scan(*a, softplus=True, stream=s),
            "selective_scan_step": lambda s: dwc.selective_scan_step(*a, softplus=True, stream=s),
            "selective_scan_bwd": lambda s: dwc.selective_scan_bwd(a[1], None, *a, softplus=True,
                                                                   stream=s),
            "residual_norm": lambda s: dwc.residual_norm(a[0], a[1], stream=s),
            "residual_norm_bwd": lambda s: dwc.residual_norm_bwd(r, h, a[0], a[1], q1, q2,
                                                                 stream=s)}


@pytest.mark.parametrize("name", ["causal_conv", "causal_conv_step", "causal_conv_bwd",
                                  "selective_scan", "selective_scan_step", "selective_scan_bwd",
                                  "residual_norm", "residual_norm_bwd"])
@pytest.mark.parametrize("handle", [False, True])
def test_on_another_stream(name, handle):
    """What a call allocates there is not memory that the current stream
    still reads, and outputs outlive their readers here."""
    log(f"case stream {name} {handle}")
    call = calls()[name]
    want = [t.clone() if t is not None else None for t in call(None)]
    side = torch.cuda.Stream()
    sync()
    here = torch.cuda.current_stream()
    held = [torch.full((1 << n,), 7.0, device="cuda") for n in range(10, 22)]
    copies = [torch.empty_like(t) for t in held]
    sync()
    torch.cuda._sleep(20_000_000)
    for c, t in zip(copies, held):
        c.copy_(t)
    del held, t
    got = call(side.cuda_stream if handle else side)
    here.wait_stream(side)
    torch.cuda._sleep(20_000_000)
    kept = [t.clone() if t is not None else None for t in got]
    del got
    with torch.cuda.stream(side):
        over = [torch.full_like(t, 3.0) for t in want if t is not None for _ in range(3)]
    sync()
    for c in copies:
        assert (c == 7.0).all()
    for s, t in zip(kept, want):
        assert s is t is None or torch.equal(s, t)
    del over


def test_autograd_of_parts():
    """Gradients where only some inputs or outputs take part; a second
    derivative raises; an input written after the forward pass is noticed."""
    a = inputs(4, 1, 12, 10, 4, 2, F32)
    leaves = [t.clone().requires_grad_() for t in a]
    y, s1 = selective_scan(*leaves, softplus=True)
    s1.sum().backward()
    want = dwc.selective_scan_bwd(torch.zeros_like(a[0]), torch.ones_like(s1), *a, softplus=True)
    for t, g in zip(leaves, want):
        assert torch.equal(t.grad, g)
    x, w = randn(1, 2, 7, 8).requires_grad_(), randn(2, 3, 8).half().requires_grad_()
    y, s1 = causal_conv(x, w, act="silu")
    s1.sum().backward()
    assert w.grad.dtype == F16 and (w.grad == 0).all() and (x.grad[:, :5] == 0).all()
    assert (x.grad[:, 5:] == 1).all()
    x.grad = None
    r, h = residual_norm(x, x)
    h.sum().backward(retain_graph=True)
    one = x.grad.clone()
    r.sum().backward()
    assert not torch.equal(one, x.grad)
    y = rms_norm(x, gate=x)
    (g,) = torch.autograd.grad(y.sum(), x, create_graph=True)
    with pytest.raises(RuntimeError, match="differentiable once"):
        g.sum().backward()
    y, _ = causal_conv(x.detach(), w)
    with torch.no_grad():
        w.add_(1)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.sum().backward()


def test_broadcast_operands_get_summed_gradients():
    """B and C of one group given to all, by expanding."""
    a = inputs(6, 2, 15, 12, 4, 1, F32)
    leaves = [t.clone().requires_grad_() for t in a]
    B = leaves[3].expand(-1, -1, 3, -1)
    C = leaves[4].expand(-1, -1, 3, -1)
    y, _ = selective_scan(*leaves[:3], B, C, *leaves[5:], softplus=True)
    y.sum().backward()
    want = dwc.selective_scan_bwd(torch.ones_like(y), None, *a, softplus=True)
    for t, g in zip(leaves, want):
        near(t.grad, g.double(), 1e-5, "gradient")


def test_saved_state_in_place_is_counted():
    a = inputs(7, 1, 4, 8, 4, 1, F32)
    s0 = a[8]
    v = s0._version
    dwc.selective_scan_step(*a, softplus=True, out_state=s0)
    assert s0._version == v + 1
    taps = randn(1, 1, 3, 8)
    v = taps._version
    dwc.causal_conv_step(a[0], randn(2, 4, 8), None, taps, out_state=taps)
    assert taps._version == v + 1
