"""The residual norm against its definition in 64 bits.

Bounds.  u = 2^-24.  A row's sum runs over at most 32 values in a lane, then a
tree: under 64 roundings a value's path.  Squares do not cancel, so a mean of
squares is off by 65 u of itself, its square root and reciprocal by 36 u.  A
gate's sigmoid is off by (2 |g| + 6) u of itself.  Errors of r are carried by
the magnitudes that r was summed from (R below).
"""

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

from gpu_helpers import dwc, log, sync  # noqa: E402
from test_sequence_gpu import BF16, F16, F32, U, close, half_step, randn  # noqa: E402

EPS = 1e-5


def gate_of(act, gate):
    """act, its slope and the relative error of both."""
    if gate is None:
        return 1.0, 0.0, 0.0
    g = gate.double()
    s = torch.sigmoid(g)
    if act == "none":
        return g, torch.ones_like(g), 0.0
    err = (2 * g.abs() + 8) * U
    if act == "sigmoid":
        return s, s * (1 - s), err
    return g * s, s + g * s * (1 - s), err


def reference(x, y, gate, scale, w1, w2, post, pre, act, dr=None, dh=None):
    c = y.shape[-1]
    one = torch.ones(c, dtype=torch.float64, device="cuda")
    Y, W1, W2, S = y.double(), *(t.double() if t is not None else one for t in (w1, w2, scale))
    X = x.double() if x is not None else torch.zeros_like(Y)
    q1 = 1 / torch.sqrt((Y * Y).mean(-1, keepdim=True) + EPS) if post else torch.ones_like(Y[..., :1])
    a, slope, ea = gate_of(act, gate)
    yh = Y * q1
    p = yh * W1
    r = X + S * a * p
    ep = (40 * U + ea) * (S * a * p).abs() + U * r.abs()  # of r
    out = {"r": (r, ep)}
    if post:
        out["q1"] = (q1[..., 0], 36 * U * q1[..., 0])
    if pre:
        q2 = 1 / torch.sqrt((r * r).mean(-1, keepdim=True) + EPS)
        # the sum of squares sees r's error too
        eq = 36 * U + (r.abs() * ep).mean(-1, keepdim=True) * q2 * q2
        rh = r * q2
        erh = ep * q2 + (eq + U) * rh.abs()
        out["q2"] = (q2[..., 0], (eq * q2)[..., 0])
        out["h"] = (rh * W2, (erh + 2 * U * rh.abs()) * W2.abs())
    if dr is None and dh is None:
        return out
    t = dr.double() if dr is not None else torch.zeros_like(Y)
    et = torch.zeros_like(Y)
    n = 96 + y.numel() / c / 64  # roundings of a column's sum, more than there are
    if dh is not None:
        e = dh.double() * W2
        mean, mmean = (e * rh).mean(-1, keepdim=True), (e * rh).abs().mean(-1, keepdim=True)
        emean = (e.abs() * erh).mean(-1, keepdim=True) + 68 * U * mmean
        et = ((eq + 6 * U) * q2 * (e.abs() + rh.abs() * mmean) + U * t.abs()
              + q2 * (erh * mean.abs() + rh.abs() * emean))
        t = t + q2 * (e - rh * mean)
        out["dw_pre"] = ((dh.double() * rh).flatten(0, -2).sum(0),
                         (dh.double().abs() * (erh + n * U * rh.abs())).flatten(0, -2).sum(0))
        et = et + U * t.abs()
    out["dx"] = (t, et)
    rel = ea + 46 * U
    out["dgate"] = (t * S * p * slope, (et + rel * t.abs()) * (S * p).abs()
                    * (slope if isinstance(slope, float) else gate_terms(act, gate)))
    out["dscale"] = ((t * a * p).flatten(0, -2).sum(0),
                     ((et + (rel + n * U) * t.abs()) * (a * p).abs()).flatten(0, -2).sum(0))
    dp, edp = t * S * a, (et + (ea + 4 * U) * t.abs()) * (S * a).abs()
    out["dw_post"] = ((dp * yh).flatten(0, -2).sum(0),
                      ((edp + (40 + n) * U * dp.abs()) * yh.abs()).flatten(0, -2).sum(0))
    e1, ee1 = dp * W1, (edp + U * dp.abs()) * W1.abs()
    dy, edy = e1 * q1, ee1 * q1 + 40 * U * (e1 * q1).abs()
    if post:
        mean = (e1 * yh).mean(-1, keepdim=True)
        mm = (e1 * yh).abs().mean(-1, keepdim=True)
        em = (ee1 * yh.abs()).mean(-1, keepdim=True) + 110 * U * mm
        dy = dy - yh * mean * q1
        edy = edy + q1 * yh.abs() * (em + 80 * U * mm) + 2 * U * dy.abs()
    out["dy"] = (dy, edy)
    return out


def gate_terms(act, gate):
    """Magnitudes that the slope is summed from."""
    g = gate.double()
    s = torch.sigmoid(g)
    return {"none": torch.ones_like(g), "sigmoid": s, "silu": s + (g * s).abs()}[act]


def check(name, got, ref):
    want, bound = ref
    close(got, want, bound + (half_step(got.dtype, want) if got.dtype != F32 else 0), name)


SIZES = [(1, 1), (3, 2), (5, 8), (33, 24), (49, 64), (7, 100), (130, 257), (65, 512), (17, 1000),
         (9, 1031), (5, 2048), (6, 4096), (3, 5003), (4, 8192), (2, 8200), (2, 16384), (1, 40000)]
TYPES = [(F32, F32), (F32, BF16), (BF16, BF16), (F32, F16), (F16, F16)]
HOW = [("none", False, True, True, True, True), ("silu", True, True, True, True, True),
       ("sigmoid", True, False, True, True, False), ("none", True, True, False, True, True),
       ("silu", True, False, False, False, False), ("none", False, False, True, False, False)]


@pytest.mark.parametrize("rows,c", SIZES)
@pytest.mark.parametrize("xt,yt", TYPES)
def test_residual_norm(rows, c, xt, yt):
    for i, (act, gated, scaled, post, pre, weighted) in enumerate(HOW):
        log(f"case residual norm {rows} {c} {xt} {yt} {HOW[i]}")
        x = randn(1, rows, c, dtype=xt) if i != 4 else None
        y = randn(2, rows, c, dtype=yt, scale=0.7)
        gate = randn(3, rows, c, dtype=yt) if gated else None
        scale = randn(4, c, shift=0.5, scale=0.3) if scaled else None
        w1 = randn(5, c, shift=1.0, scale=0.2) if weighted and post else None
        w2 = randn(6, c, shift=1.0, scale=0.2) if weighted and pre else None
        dr = randn(7, rows, c, dtype=xt if x is not None else yt) if i != 2 else None
        dh = randn(8, rows, c, dtype=yt) if pre else None
        kw = dict(gate=gate, scale=scale, w_post=w1, w_pre=w2, post=post, pre=pre, act=act)
        ref = reference(x, y, gate, scale, w1, w2, post, pre, act, dr, dh)
        r, h, q1, q2 = dwc.residual_norm(x, y, eps=EPS, **kw)
        grads = dwc.residual_norm_bwd(dr, dh, x, y, q1, q2, **kw)
        sync()
        assert (h is None) == (q2 is None) == (not pre) and (q1 is None) == (not post)
        for name, got in zip(("r", "h", "q1", "q2", "dx", "dy", "dgate", "dscale", "dw_post",
                              "dw_pre"), (r, h, q1, q2) + grads):
            if got is not None:
                check(name, got, ref[name])
        for got, t in zip(grads, (x, y, gate, scale, w1, w2)):
            assert (got is None) == (t is None)
        for s, t in zip(dwc.residual_norm_bwd(dr, dh, x, y, q1, q2, **kw), grads):
            assert s is t is None or torch.equal(s, t)


def test_strides_types_and_ranks():
    big = randn(9, 12, 200, dtype=BF16)
    for lo in (16, 3):
        x, y, g = big[:, lo:lo + 48], big[:, lo + 48:lo + 96], big[:, lo + 96:lo + 144]
        w = randn(10, 48, dtype=F16, shift=1.0)
        args = dict(gate=g, w_post=w, scale=w, act="silu")
        r, h, q1, q2 = dwc.residual_norm(x, y, **args)
        ref = reference(x, y, g, w, w, None, True, True, "silu", x, y)
        grads = dwc.residual_norm_bwd(x, y, x, y, q1, q2, **args)
        for name, got in zip(("r", "h", "dx", "dy", "dgate", "dscale", "dw_post"),
                             (r, h) + grads[:5]):
            check(name, got, ref[name])
    x4 = randn(11, 2, 3, 5, 64, dtype=F16)
    r, h, q1, q2 = dwc.residual_norm(x4, x4)
    assert r.shape == h.shape == x4.shape and q1.shape == q2.shape == x4.shape[:-1]
    r2, h2, _, _ = dwc.residual_norm(x4.view(-1, 64), x4.view(-1, 64))
    assert torch.equal(r2, r.view(-1, 64)) and torch.equal(h2, h.view(-1, 64))


def test_by_differences():
    x, y, g = randn(1, 3, 10), randn(2, 3, 10), randn(3, 3, 10)
    s, w1, w2 = (randn(i, 10, shift=1.0) for i in (4, 5, 6))
    dr, dh = randn(7, 3, 10), randn(8, 3, 10)
    _, _, q1, q2 = dwc.residual_norm(x, y, g, s, w1, w2, eps=EPS, act="silu")
    got = dwc.residual_norm_bwd(dr, dh, x, y, q1, q2, g, s, w1, w2, act="silu")
    args, step = [t.double() for t in (x, y, g, s, w1, w2)], 1e-5

    def f():
        ref = reference(*args, True, True, "silu")
        return ((ref["r"][0] * dr.double()).sum() + (ref["h"][0] * dh.double()).sum()).item()

    for a, d in zip(args, got):
        for i in range(0, a.numel(), 3):
            flat, old = a.view(-1), a.view(-1)[i].item()
            flat[i] = old + step
            up = f()
            flat[i] = old - step
            down = f()
            flat[i] = old
            # step^2 of the third derivative and 64-bit noise / step
            got_i = d.view(-1)[i].item()
            assert abs((up - down) / (2 * step) - got_i) < 2e-5 * (1 + abs(got_i))


def test_empty_rows_and_zero_rows():
    y = torch.empty(0, 16, device="cuda", dtype=BF16)
    r, h, q1, q2 = dwc.residual_norm(y, y)
    assert r.shape == h.shape == (0, 16) and q1.shape == (0,)
    w = randn(1, 16)
    g = dwc.residual_norm_bwd(y, y, y, y, q1, q2, scale=w, w_post=w, w_pre=w)
    assert all((t == 0).all() for t in g[3:])
    y = torch.zeros(4, 16, device="cuda")
    r, h, q1, q2 = dwc.residual_norm(y, y)
    assert (r == 0).all() and (h == 0).all() and torch.isfinite(q1).all()


def test_a_row_does_not_reach_another():
    x, y = randn(1, 20, 300, dtype=BF16), randn(2, 20, 300, dtype=BF16)
    clean = dwc.residual_norm(x, y)
    y[7, 5], x[9, 0] = float("nan"), float("inf")
    got = dwc.residual_norm(x, y)
    keep = torch.ones(20, dtype=torch.bool, device="cuda")
    keep[7] = keep[9] = False
    for s, t in zip(got, clean):
        assert torch.equal(s[keep], t[keep])
    assert torch.isnan(got[1][7]).all()


def test_refusals():
    x = randn(1, 4, 8)
    w = randn(2, 8)
    for bad, args, kw in [
            (ValueError, (x, x[:2]), {}), (TypeError, (x.half(), x), {}),
            (TypeError, (x, x, x.half()), {}), (ValueError, (x, x, x[:, :4]), {}),
            (ValueError, (x, x, None, w[:4]), {}), (TypeError, (x, x, None, w, w.half()), {}),
            (ValueError, (x, x, None, None, w), dict(post=False)),
            (ValueError, (x, x, None, None, None, w), dict(pre=False)),
            (ValueError, (x, x, x), dict(act="relu")), (ValueError, (x, x.t().contiguous().t()), {}),
            (dwc.DwcError, (x, x), dict(eps=-1.0)), (TypeError, (x, None), {})]:
        with pytest.raises(bad):
            dwc.residual_norm(*args, **kw)
    r, h, q1, q2 = dwc.residual_norm(x, x)
    for args, kw in [((None, None, x, x, q1, q2), {}), ((x, x, x, x, q1, q2), dict(pre=False)),
                     ((x, x, x, x, q1[:2], q2), {}), ((x[:2], x, x, x, q1, q2), {})]:
        with pytest.raises(ValueError):
            dwc.residual_norm_bwd(*args, **kw)
    with pytest.raises(TypeError):
        dwc.residual_norm_bwd(x, x, x, x, None, q2)


@pytest.mark.parametrize("c", [64, 777, 9000])
def test_gradients_of_the_sum_alone(c):
    """Without a gradient of h its norm's values are not needed."""
    log(f"case residual norm without dh, {c}")
    x, y, dr = (randn(30 + i, 5, c) for i in range(3))
    w = randn(33, c)
    r, h, q1, q2 = dwc.residual_norm(x, y, w_post=w, w_pre=w)
    want = dwc.residual_norm_bwd(dr, torch.zeros_like(dr), x, y, q1, q2, w_post=w, w_pre=w)
    for q in (q2, None):
        got = dwc.residual_norm_bwd(dr, None, x, y, q1, q, w_post=w, w_pre=w)
        for s, t in zip(got, want):
            assert s is t is None or (s == t).all()
