"""The chunked gated delta rule and its gradients against the rule token by
token in 64 bits (and autograd's gradient of it), and against differences.

Bounds, as 2-norms of a whole output.  The kernels multiply pairs of fp16
numbers that hold 22 bits, so a product is off by about 2^-23 of its size
and a chunk's chain of five products, with the triangular solve between
them, by under 2^-19; states forget at the tested decays, so errors of
chunks do not pile up.  F = 1e-5 > 5 * 2^-19 covers fp32 outputs.  Outputs
of 16 bits add half a step of their type; in bf16 the last products of o, dk
take one fp16 number an operand, 2^-12 each.
"""

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

from gpu_helpers import dwc, log, sync  # noqa: E402
from test_sequence_gpu import (BF16, F16, F32, delta_inputs, half, randn, rel)  # noqa: E402

F = 1e-5
TOL = {F32: F, F16: half(F16) + F, BF16: half(BF16) + 2 * 2.0 ** -12 + F}


def reference(q, k, v, g, beta, s0, lengths=None, scale=None):
    """(o, s1) in 64 bits, differentiable."""
    b, n, hv, dv = v.shape
    hk, dk = q.shape[2:]
    scale = dk ** -0.5 if scale is None else scale
    q, k = (t.repeat_interleave(hv // hk, 2) for t in (q, k))
    a, s, os = g.exp(), s0, []
    for t in range(n):
        dec = s * a[:, t, :, None, None]
        u = beta[:, t, :, None] * (v[:, t] - (dec * k[:, t, :, :, None]).sum(2))
        new = dec + k[:, t, :, :, None] * u[:, :, None, :]
        o = scale * (new * q[:, t, :, :, None]).sum(2)
        if lengths is not None:
            live = (t < lengths)[:, None, None]
            new, o = torch.where(live[..., None], new, s), torch.where(live, o, 0.0)
        s = new
        os.append(o)
    return (torch.stack(os, 1) if os else torch.zeros_like(v)), s


def wanted(a, dout, ds1, lengths=None, scale=None):
    b, n, hv, dv = a[2].shape
    s0 = a[5] if a[5] is not None else torch.zeros(b, hv, a[0].shape[3], dv, device="cuda")
    leaves = [t.double().clone().requires_grad_() for t in list(a[:5]) + [s0]]
    o, s1 = reference(*leaves, lengths, scale)
    grads = torch.autograd.grad([o, s1], leaves, [dout.double(), ds1.double()],
                                allow_unused=True)
    grads = [torch.zeros_like(x) if d is None else d for d, x in zip(grads, leaves)]
    return o.detach(), s1.detach(), grads


def check(a, lengths=None, scale=None, seed=50, state_grad=True):
    dtype = a[0].dtype
    b, n, hv, dv = a[2].shape
    dk = a[0].shape[3]
    dout = randn(seed, b, n, hv, dv, dtype=dtype)
    ds1 = randn(seed + 1, b, hv, dk, dv, scale=0.1) if state_grad else None
    o, s1 = dwc.delta_rule(*a, lengths=lengths, scale=scale)
    grads = dwc.delta_rule_bwd(dout, ds1, *a, lengths=lengths, scale=scale)
    sync()
    zero = torch.zeros(b, hv, dk, dv, device="cuda")
    clean = [torch.nan_to_num(t, 0.0, 0.0, 0.0) for t in a[:5]] + [a[5]]
    wo, ws, wg = wanted(clean, dout, zero if ds1 is None else ds1, lengths, scale)
    names = ("dq", "dk", "dv", "dg", "dbeta", "ds0")
    for name, got, want in [("o", o, wo), ("s1", s1, ws)] + list(zip(names, grads, wg)):
        if got is None:
            assert name == "ds0" and a[5] is None
            continue
        assert torch.isfinite(got).all(), name
        r = rel(got, want)
        log(f"{name} {r:.3g}")
        assert r < (TOL[got.dtype]), (name, r)
    if lengths is not None:
        for i, m in enumerate(lengths.tolist()):
            for t in (o,) + grads[:5]:
                assert not t[i, max(0, m):].any()
    return o, s1, grads


SHAPES = [(1, 1, 1, 1, 1, 1), (2, 2, 1, 1, 8, 4), (1, 63, 1, 2, 16, 16), (1, 64, 2, 2, 64, 64),
          (2, 65, 1, 3, 100, 75), (1, 130, 2, 4, 128, 128), (3, 200, 2, 2, 96, 72),
          (1, 333, 1, 1, 33, 130), (2, 64, 1, 2, 128, 7), (1, 700, 1, 2, 64, 64)]


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("shape", SHAPES)
def test_delta_chunked(dtype, shape):
    log(f"case delta {dtype} {shape}")
    check(delta_inputs(sum(shape), *shape, dtype, state=True))
    if shape[1] in (65, 64, 200):
        check(delta_inputs(sum(shape), *shape, dtype, state=False), state_grad=False)


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
def test_delta_lengths_and_masked_places(dtype):
    log(f"case delta lengths {dtype}")
    a = list(delta_inputs(7, 6, 150, 2, 4, 40, 24, dtype))
    lengths = torch.tensor([0, 1, 64, 65, 150, 149], dtype=torch.int32, device="cuda")
    a[3], a[4] = a[3].clone(), a[4].clone()
    for i, m in enumerate(lengths.tolist()):
        for t in a[:3]:
            t[i, m:] = float("nan")
        a[3][i, m:], a[4][i, m:] = float("nan"), float("inf")
    o, s1, grads = check(a, lengths)
    assert torch.equal(s1[0], a[5][0])
    # lengths outside 0..l act as the nearest of them
    a = delta_inputs(8, 2, 70, 1, 1, 16, 16, dtype)
    far = torch.tensor([-5, 1000], dtype=torch.int32, device="cuda")
    near = torch.tensor([0, 70], dtype=torch.int32, device="cuda")
    for s, t in zip(dwc.delta_rule(*a, lengths=far), dwc.delta_rule(*a, lengths=near)):
        assert torch.equal(s, t)


def test_delta_strong_and_no_decay():
    a = list(delta_inputs(9, 1, 150, 1, 2, 32, 32, F32))
    a[3] = torch.zeros_like(a[3])  # nothing is forgotten
    check(a)
    a[3] = torch.full_like(a[3], -30.0)  # everything is
    o, s1 = dwc.delta_rule(*a)
    wo, ws = reference(*(t.double() for t in a))
    assert rel(o, wo) < F and rel(s1, ws) < F
    a[3][:, 70] = -float("inf")
    a[3][:, 71] = torch.finfo(F32).min
    o, s1 = dwc.delta_rule(*a)
    wo, ws = reference(*(t.double() for t in a))
    assert rel(o, wo) < F and rel(s1, ws) < F
    for t in dwc.delta_rule_bwd(a[2], None, *a):
        assert torch.isfinite(t).all()


def test_delta_beta_zero_and_scales():
    a = list(delta_inputs(10, 1, 100, 1, 2, 48, 40, F32))
    a[4] = a[4].clone()
    a[4][:, 10:40] = 0.0  # tokens that write nothing still have a gradient of beta
    check(a, scale=0.7)
    big = [a[0] * 2.0 ** 40, a[1], a[2] * 2.0 ** -30, a[3], a[4], a[5] * 2.0 ** -30]
    check(big)  # scales of operands do not matter
    zero = [torch.zeros_like(t) for t in a]
    check(zero)


def test_delta_by_differences():
    """Every gradient against central differences of the 64-bit rule."""
    a = [t.double() for t in delta_inputs(11, 1, 70, 1, 2, 6, 5, F32)]
    dout, ds1 = randn(12, 1, 70, 2, 5), randn(13, 1, 2, 6, 5)
    got = dwc.delta_rule_bwd(dout, ds1, *(t.float() for t in a))

    def f():
        o, s1 = reference(*a)
        return ((o * dout).sum() + (s1 * ds1).sum()).item()

    step = 1e-6
    a = [t.contiguous() for t in a]
    for x, d in zip(a, got):
        flat = x.view(-1)
        for i in range(0, flat.numel(), max(1, flat.numel() // 5)):
            old = flat[i].item()
            flat[i] = old + step
            up = f()
            flat[i] = old - step
            down = f()
            flat[i] = old
            num = (up - down) / (2 * step)
            # 64-bit noise of values under 1e2 over the step: 1e-8; the fp32
            # gradient: F of its norm
            assert abs(num - d.contiguous().view(-1)[i].item()) < 1e-7 + F * d.norm().item()


def test_delta_steps_continue_a_prompt():
    """A prompt in chunks, then tokens one by one, as the whole at once."""
    a = delta_inputs(14, 2, 100, 2, 4, 64, 64, F32)
    o, s1 = dwc.delta_rule(*a)
    head = [t[:, :90] for t in a[:5]]
    p, s = dwc.delta_rule(*head, a[5])
    parts = [p]
    for t in range(90, 100):
        p, s = dwc.delta_rule_step(*(x[:, t:t + 1] for x in a[:5]), s, out_state=s)
        parts.append(p)
    assert rel(torch.cat(parts, 1), o.double()) < 2 * F and rel(s, s1.double()) < 2 * F


def test_delta_empty_same_bits_streams_and_refusals():
    a = list(delta_inputs(15, 2, 0, 1, 1, 16, 8, F32))
    o, s1 = dwc.delta_rule(*a)
    assert o.shape == (2, 0, 1, 8) and torch.equal(s1, a[5])
    ds = randn(16, 2, 1, 16, 8)
    assert torch.equal(dwc.delta_rule_bwd(a[2], ds, *a)[5], ds)
    a = delta_inputs(17, 2, 300, 2, 4, 128, 128, BF16)
    do = randn(18, 2, 300, 4, 128, dtype=BF16)
    first = dwc.delta_rule(*a) + dwc.delta_rule_bwd(do, None, *a)
    sync()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    again = dwc.delta_rule(*a, stream=side) + dwc.delta_rule_bwd(do, None, *a, stream=side)
    side.synchronize()
    for s, t in zip(first, again):
        assert torch.equal(s, t)
    with pytest.raises(dwc.DwcError) as err:
        b = delta_inputs(19, 1, 4, 1, 1, 160, 8, F32)
        dwc.delta_rule(*b)
    assert err.value.status == 2
    with pytest.raises(ValueError):
        dwc.delta_rule_bwd(do[:, :5], None, *a)
    with pytest.raises(ValueError):
        dwc.delta_rule_bwd(do, ds, *a)
    with pytest.raises(TypeError):
        dwc.delta_rule(*a, lengths=torch.ones(2, device="cuda"))
