"""The selective scan against its definition in 64 bits, token by token.

Bounds are carried beside the values.  u = 2^-24.  A step dt is off by
u |x| slope (its sum with the bias) and (2 |x| + 14) u of itself (softplus:
an exp whose argument is rounded twice, a logarithm, a reciprocal and five
more roundings).  A decay exp(dt A) is off by dt's error times |A| and
(3 |dt A| + 4) u of itself; chunks multiply their decays over a chunk, which
adds 4 u for each chunk, less than that for each token.  States, their
gradients and every sum get the errors of what they are made of and a
rounding for each term; a sum over c channels or tokens at most 96 of them
(in a lane at most 32, then trees and 64 partial sums, and one for each 64
rows of partial sums).  Below 2^-126 the exp instruction gives 0, so that a
decay is off by up to that whatever it is itself; products of that size are
off by half of 2^-149 each, of which a value sees fewer than 2^23 (TINY covers
both).
"""

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

from gpu_helpers import dwc, log, sync  # noqa: E402
from test_sequence_gpu import BF16, F16, F32, U, close, half_step, randn  # noqa: E402

TINY = 2.0 ** -126
NAMES = ("y", "s1", "du", "ddelta", "dA", "dB", "dC", "dD", "dz", "dbias", "ds0")


def inputs(seed, b, l, d, n, g, dtype, gate=True, state=True, soft=True, strided=False):
    """The arguments of selective_scan, softplus left out."""
    u = randn(seed, b, l, d, dtype=dtype)
    delta = randn(seed + 1, b, l, d, dtype=dtype, scale=0.5)
    if not soft:
        delta = delta.abs() * 0.1
    mixed = randn(seed + 2, b, l, 2 * g * n + 3, dtype=dtype)
    B, C = (mixed[..., i:i + g * n].unflatten(-1, (g, n)) for i in (1, 2 + g * n))
    if not strided:
        B, C = B.contiguous(), C.contiguous()
    A = -(torch.arange(1, n + 1) * torch.exp(randn(seed + 3, d, n).cpu() * 0.1)).cuda()
    z = randn(seed + 4, b, l, 2 * d, dtype=dtype)[..., d:] if gate else None
    D, bias = randn(seed + 5, d), randn(seed + 6, d) - 2.0 if soft else None
    s0 = randn(seed + 7, b, d, n, scale=0.5) if state else None
    return [u, delta, A, B, C, D, z, bias, s0]


def reference(a, lens, soft, dy=None, ds1=None):
    """{name: (value, bound)}"""
    u, delta, A, B, C, D, z, bias, s0 = (t.double() if t is not None else None for t in a)
    b, l, d = u.shape
    n, g = A.shape[1], B.shape[2]
    zero = torch.zeros(b, d, n, dtype=torch.float64, device="cuda")
    each = lambda t: t.repeat_interleave(d // g, 1)  # noqa: E731
    live = torch.ones(b, l, 1, dtype=torch.bool, device="cuda")
    if lens is not None:
        ends = torch.tensor(lens, device="cuda").clamp(0, l)
        live = (torch.arange(l, device="cuda") < ends[:, None])[..., None]
    pick = lambda t: torch.where(live if t.dim() == 3 else live[..., None], t, 0.0)  # noqa: E731
    u, delta, B, C = (pick(t) for t in (u, delta, B, C))
    x = delta + (bias if bias is not None else 0.0)
    if soft:
        dt, slope = torch.logaddexp(x, torch.zeros_like(x)), torch.sigmoid(x)
        edt = U * x.abs() * slope + (2 * x.abs() + 14) * U * dt
    else:
        dt, slope, edt = x, torch.ones_like(x), U * x.abs()
    dt, edt = pick(dt), pick(edt)
    silu = esilu = None
    if z is not None:
        z = pick(z)
        sig = torch.sigmoid(z)
        silu, dsilu = z * sig, sig + z * sig * (1 - sig)
        esilu = (2 * z.abs() + 8) * U
    Dv = D if D is not None else torch.zeros(d).double().cuda()
    h, m, e = (s0 if s0 is not None else zero), (s0.abs() if s0 is not None else zero), zero
    hs, ms, es, decays, deltas = [h], [m], [e], [], []
    o, mo, eo = (torch.zeros_like(u) for _ in range(3))
    for t in range(l):
        s, es_ = dt[:, t, :, None], edt[:, t, :, None]
        k = torch.exp(s * A)
        ek = (es_ * A.abs() + (3 * (s * A).abs() + 8) * U) * k + TINY
        bb, cc, uu = each(B[:, t]), each(C[:, t]), u[:, t, :, None]
        into = s * uu * bb
        e = k * e + ek * m + TINY + (es_ * (uu * bb).abs() + 4 * U * into.abs())
        h, m = k * h + into, k * m + into.abs()
        e = e + 2 * U * m
        o[:, t] = (cc * h).sum(-1) + Dv * u[:, t]
        mo[:, t] = (cc.abs() * m).sum(-1) + (Dv * u[:, t]).abs()
        eo[:, t] = (cc.abs() * e).sum(-1) + (n + 3) * U * mo[:, t]
        hs.append(h), ms.append(m), es.append(e), decays.append(k), deltas.append(ek)
    out = {"s1": (h, e)}
    if z is None:
        out["y"] = (pick(o), eo)
    else:
        out["y"] = (pick(o * silu), eo * silu.abs() + (esilu + U) * mo * silu.abs())
    if dy is None:
        return out
    dy = pick(dy.double())
    go, ego, dz, edz = dy, 0 * dy, None, None
    if z is not None:
        go, ego = dy * silu, dy.abs() * silu.abs() * (esilu + U)
        dz = dy * o * dsilu
        edz = dy.abs() * (eo * dsilu.abs() + mo * (esilu + 6 * U) * (sig + (z * sig).abs()))
    G = ds1.double() if ds1 is not None else zero
    M, E = G.abs(), zero
    du, ddt, edu, eddt = (torch.zeros_like(u) for _ in range(4))
    dB, dC, eB, eC = (torch.zeros_like(B) for _ in range(4))
    dA, eA = torch.zeros_like(A), torch.zeros_like(A)
    red = lambda t: t.unflatten(1, (g, d // g)).sum(2)  # noqa: E731
    long = 96 + b * l / 32 / 64
    for t in reversed(range(l)):
        s, es_ = dt[:, t, :, None], edt[:, t, :, None]
        bb, cc, uu = each(B[:, t]), each(C[:, t]), u[:, t, :, None]
        gg, eg = go[:, t, :, None], ego[:, t, :, None]
        # G: into h_t; M: its magnitude; E: its bound
        E = E + cc.abs() * eg + U * (M + (cc * gg).abs())
        G, M = G + cc * gg, M + (cc * gg).abs()
        dC[:, t] = red(gg * hs[t + 1])
        eC[:, t] = red(gg.abs() * es[t + 1] + (eg + long * U * gg.abs()) * ms[t + 1])
        w = s * uu
        dB[:, t] = red(G * w)
        eB[:, t] = red(E * w.abs() + M * (es_ * uu.abs() + long * U * w.abs()))
        gb, mgb = (G * bb).sum(-1), (M * bb.abs()).sum(-1)
        egb = (E * bb.abs()).sum(-1) + (n + 2) * U * mgb
        k, ek = decays[t], deltas[t]
        q, mq = G * k * hs[t], M * k * ms[t]
        eq = E * k * ms[t] + M * k * es[t] + ek * M * ms[t] + 4 * U * mq + TINY
        ddt[:, t] = (A * q).sum(-1) + u[:, t] * gb
        eddt[:, t] = ((A.abs() * eq).sum(-1) + (n + 6) * U * (A.abs() * mq).sum(-1)
                      + u[:, t].abs() * (egb + 2 * U * mgb))
        du[:, t] = dt[:, t] * gb + Dv * go[:, t]
        edu[:, t] = (edt[:, t] * mgb + dt[:, t] * (egb + U * mgb) + Dv.abs() * ego[:, t]
                     + 2 * U * (Dv * go[:, t]).abs())
        dA += (s * q).sum(0)
        eA += (es_ * mq + s * (eq + long * U * mq)).sum(0)
        E, G, M = E * k + (ek + U * k) * M + TINY, G * k, M * k
    es_ = (2 * x.abs() + 8) * U + (U * x.abs() if soft else 0)  # of slope, and through x
    mddt = ddt.abs() + eddt
    dx, edx = ddt * slope, eddt * slope + (es_ if soft else U) * mddt * slope
    dx, edx = pick(dx), pick(edx)
    out.update(du=(pick(du), pick(edu)), ddelta=(dx, edx), dA=(dA, eA), dB=(pick(dB), eB),
               dC=(pick(dC), eC),
               dD=((go * u).sum((0, 1)), (ego * u.abs() + long * U * (go * u).abs()).sum((0, 1))),
               dz=(dz, edz), dbias=(dx.sum((0, 1)), (edx + long * U * mddt * slope).sum((0, 1))),
               ds0=(G, E))
    return out


def check(name, got, ref):
    want, bound = ref
    close(got, want, bound + (half_step(got.dtype, want) if got.dtype != F32 else 0), name)


CASES = [  # b, l, d, n, g, lengths, gate, state, softplus
    (1, 1, 1, 1, 1, None, True, True, True), (2, 1, 64, 16, 1, None, True, True, True),
    (1, 7, 3, 4, 1, None, False, False, True), (2, 8, 65, 5, 1, None, True, False, False),
    (1, 33, 128, 16, 1, None, True, True, True), (2, 40, 130, 8, 2, None, True, True, True),
    (1, 100, 96, 16, 3, None, False, True, True), (1, 65, 66, 17, 2, None, True, True, True),
    (1, 31, 40, 64, 1, None, True, False, True), (1, 34, 24, 256, 1, None, True, True, True),
    (4, 70, 72, 16, 1, [70, 0, 1, 33], True, True, True), (3, 40, 20, 33, 2, [64, -1, 8], True, True, True),
    (2, 300, 260, 16, 1, [300, 128], True, True, True), (2, 9, 129, 12, 1, None, False, False, False)]


def run_case(b, l, d, n, g, lens, gate, state, soft, dtype, strided=False):
    a = inputs(10, b, l, d, n, g, dtype, gate, state, soft, strided)
    dy = randn(1, b, l, d, dtype=dtype)
    ds1 = randn(2, b, d, n) if state else None
    lengths = torch.tensor(lens, dtype=torch.int32, device="cuda") if lens else None
    ref = reference(a, lens, soft, dy, ds1)
    if lens:  # nothing past a length is read
        for i, m in enumerate(lens):
            for t in (a[0], a[1], a[3], a[4], a[6], dy):
                if t is not None:
                    t[i, max(m, 0):] = float("nan")
    y, s1 = dwc.selective_scan(*a, lengths=lengths, softplus=soft)
    grads = dwc.selective_scan_bwd(dy, ds1, *a, lengths=lengths, softplus=soft)
    sync()
    for name, got in zip(NAMES, (y, s1) + grads):
        if got is not None:
            check(name, got, ref[name])
    for got, t in zip(grads, a):
        assert (got is None) == (t is None)
    ys, ss = dwc.selective_scan_step(*a, lengths=lengths, softplus=soft)
    check("y by token", ys, ref["y"])
    check("s1 by token", ss, ref["s1"])
    again = dwc.selective_scan_bwd(dy, ds1, *a, lengths=lengths, softplus=soft)
    for s, t in zip(again, grads):
        assert s is t is None or torch.equal(s, t)


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("b,l,d,n,g,lens,gate,state,soft", CASES)
def test_selective_scan(b, l, d, n, g, lens, gate, state, soft, dtype):
    log(f"case scan {b} {l} {d} {n} {g} {lens} {gate} {state} {soft} {dtype}")
    run_case(b, l, d, n, g, lens, gate, state, soft, dtype)


@pytest.mark.parametrize("b,l,d,n,g,lens", [(2, 35, 70, 16, 2, None), (2, 20, 33, 7, 1, [20, 11])])
def test_strided_operands(b, l, d, n, g, lens):
    """B and C inside one tensor at odd offsets, z in the half of another."""
    log(f"case scan strided {b} {l} {d} {n}")
    run_case(b, l, d, n, g, lens, True, True, True, F16, strided=True)


def test_few_arguments():
    """No D, no bias, no gate, no state; a gradient of the state alone."""
    a = inputs(3, 2, 20, 10, 4, 1, F32, gate=False, state=False, soft=False)
    a[5] = None
    dy, ds1 = torch.zeros_like(a[0]), randn(4, 2, 10, 4)
    ref = reference(a, None, False, dy, ds1)
    y, s1 = dwc.selective_scan(*a[:5])
    got = (y, s1) + dwc.selective_scan_bwd(dy, ds1, *a[:5])
    for name, t in zip(NAMES, got):
        if t is not None:
            check(name, t, ref[name])


def test_pieces_give_the_whole():
    a = inputs(5, 2, 90, 30, 16, 1, BF16, state=False)
    whole, end = dwc.selective_scan(*a, softplus=True)
    ref = reference(a, None, True)
    state, out = torch.zeros_like(end), []
    for lo, hi in ((0, 1), (1, 2), (2, 40), (40, 43), (43, 90)):
        p = [t[:, lo:hi] if t is not None and i in (0, 1, 3, 4, 6) else t for i, t in enumerate(a)]
        if hi - lo > 5:
            y, state = dwc.selective_scan(*p[:8], state, softplus=True)
        else:
            y, s1 = dwc.selective_scan_step(*p[:8], state, softplus=True, out_state=state)
            assert s1 is state
        out.append(y)
    check("y in pieces", torch.cat(out, 1), ref["y"])
    check("s1 in pieces", state, ref["s1"])
    check("y whole", whole, ref["y"])


def test_small_steps_keep_their_bits():
    """softplus far below zero: y is the step itself (A = 0, B = C = u = 1)."""
    x = torch.linspace(-80.0, 30.0, 4096, device="cuda").view(1, 1, -1)
    one = torch.ones(1, 1, 1, 1, device="cuda")
    A = torch.zeros(4096, 1, device="cuda")
    want = torch.logaddexp(x.double(), torch.zeros_like(x).double())
    for f in (dwc.selective_scan, dwc.selective_scan_step):
        y, _ = f(torch.ones_like(x), x, A, one, one, softplus=True)
        close(y, want, (2 * x.double().abs() + 16) * U * want, "softplus")


def test_long_decays():
    """Decays that forget at once and ones that keep everything, over many
    chunks; steps of zero leave the state as it is."""
    a = inputs(7, 1, 500, 8, 16, 1, F32)
    a[2][:4] *= 100.0
    a[2][4:] *= 1e-4
    a[1][:, 100:200] = -1e4  # softplus 0
    dy, ds1 = randn(8, 1, 500, 8), randn(9, 1, 8, 16)
    ref = reference(a, None, True, dy, ds1)
    got = dwc.selective_scan(*a, softplus=True)
    got += dwc.selective_scan_bwd(dy, ds1, *a, softplus=True)
    for name, t in zip(NAMES, got):
        check(name, t, ref[name])


def test_gradient_by_differences():
    a = inputs(9, 1, 5, 4, 3, 2, F32)
    dy, ds1 = randn(10, 1, 5, 4), randn(11, 1, 4, 3)
    got = dwc.selective_scan_bwd(dy, ds1, *a, softplus=True)
    args, step = [t.double().contiguous() for t in a], 1e-5

    def f():
        r = reference(args, None, True)
        return ((r["y"][0] * dy.double()).sum() + (r["s1"][0] * ds1.double()).sum()).item()

    for t, g in zip(args, got):
        for i in range(t.numel()):
            flat, old = t.view(-1), t.view(-1)[i].item()
            flat[i] = old + step
            up = f()
            flat[i] = old - step
            down = f()
            flat[i] = old
            # step^2 of the third derivative and 64-bit noise / step: < 1e-6 of 1 + |g|
            got_i = g.reshape(-1)[i].item()
            assert abs((up - down) / (2 * step) - got_i) < 2e-5 * (1 + abs(got_i))


def test_empty():
    a = inputs(12, 2, 0, 8, 4, 1, BF16)
    y, s1 = dwc.selective_scan(*a, softplus=True)
    assert y.shape == (2, 0, 8) and torch.equal(s1, a[8])
    ds1 = randn(1, 2, 8, 4)
    g = dwc.selective_scan_bwd(y, ds1, *a, softplus=True)
    assert torch.equal(g[8], ds1) and all((t == 0).all() for t in g[:8])
    a = inputs(12, 0, 5, 8, 4, 1, BF16)
    y, s1 = dwc.selective_scan(*a, softplus=True)
    g = dwc.selective_scan_bwd(y, None, *a, softplus=True)
    assert y.shape == (0, 5, 8) and s1.shape == (0, 8, 4)
    assert (g[2] == 0).all() and (g[5] == 0).all() and (g[7] == 0).all()


def test_far_offsets():
    """Tokens more than 2^32 bytes apart."""
    a = inputs(13, 1, 3, 64, 16, 1, BF16)
    far = list(a)
    for i in (0, 1, 6):
        t = torch.empty_strided((1, 3, 64), (0, (1 << 31) + 64, 1), dtype=BF16, device="cuda")
        far[i] = t.copy_(a[i])
    for s, t in zip(dwc.selective_scan(*far, softplus=True),
                    dwc.selective_scan(*a, softplus=True)):
        assert torch.equal(s, t)
    for s, t in zip(dwc.selective_scan_bwd(far[0], None, *far, softplus=True),
                    dwc.selective_scan_bwd(a[0], None, *a, softplus=True)):
        assert torch.equal(s, t)


def test_infinities_stay_in_their_channel():
    """A channel with an infinite input, a NaN in a live token: other channels
    and earlier tokens do not see it."""
    a = inputs(14, 1, 50, 70, 16, 1, F32)
    clean, _ = dwc.selective_scan(*a, softplus=True)
    a[0][0, 30, 5] = float("inf")
    a[0][0, 10, 69] = float("nan")
    y, _ = dwc.selective_scan(*a, softplus=True)
    ok = torch.ones(50, 70, dtype=torch.bool, device="cuda")
    ok[30:, 5] = ok[10:, 69] = False
    assert torch.equal(y[0][ok], clean[0][ok]) and not torch.isfinite(y[0][~ok]).any()


def test_refusals():
    a = inputs(15, 2, 5, 8, 4, 2, F32)
    names = ("u", "delta", "A", "B", "C", "D", "z", "delta_bias", "s0")

    def call(**ch):
        k = dict(zip(names, a))
        k.update(ch)
        return dwc.selective_scan(**k)

    u, delta, A, B, C, D, z, bias, s0 = a
    for bad, ch in [
            (ValueError, dict(u=u[0])), (ValueError, dict(delta=delta[:, :4])),
            (TypeError, dict(delta=delta.half())), (ValueError, dict(A=A.t())),
            (ValueError, dict(A=A[:4])), (TypeError, dict(A=A.half())),
            (ValueError, dict(B=B[:, :, :1])), (ValueError, dict(C=C[..., :3])),
            (ValueError, dict(B=B[:, :, 0])), (ValueError, dict(B=B.transpose(2, 3))),
            (TypeError, dict(B=B.half())), (ValueError, dict(D=D[:4])), (TypeError, dict(D=D.half())),
            (ValueError, dict(z=z[..., :4])), (TypeError, dict(z=z.half())),
            (ValueError, dict(delta_bias=bias[:1])), (ValueError, dict(s0=s0[:1])),
            (TypeError, dict(s0=s0.half())),
            (TypeError, dict(lengths=torch.zeros(2, device="cuda"))),
            (ValueError, dict(lengths=torch.zeros(1, dtype=torch.int32, device="cuda"))),
            (TypeError, dict(u=None))]:
        with pytest.raises(bad):
            call(**ch)
    with pytest.raises(dwc.DwcError):  # d no multiple of g
        call(B=B.repeat(1, 1, 2, 1)[:, :, :3].contiguous(), C=C.repeat(1, 1, 2, 1)[:, :, :3].contiguous())
    with pytest.raises(ValueError):
        dwc.selective_scan_step(*a, out_state=s0[:1])
    with pytest.raises(ValueError):
        dwc.selective_scan_bwd(u[:, :4], None, *a)
    assert torch.isfinite(call(softplus=True)[0]).all()
