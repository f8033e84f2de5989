"""The short causal convolution against a plain formulation in 64 bits.

Bounds.  u = 2^-24.  pre is a sum of K products and the bias: off by at most
(K + 2) u of its terms' magnitudes M.  sigmoid(p) is made of an exp (its
argument rounded twice: 2 |p| u, itself 1 ulp = 2 u), a sum and a reciprocal
(1 ulp): off by (2 |p| + 6) u of itself.  |silu'| <= 1.1 and |silu''| <= 0.5
carry pre's error on.
"""

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

from gpu_helpers import dwc, log, sync  # noqa: E402
from test_sequence_gpu import BF16, F16, F32, U, close, half_step, randn  # noqa: E402


def reference(x, w, bias, s0, lens, silu, dy=None, ds1=None):
    """Outputs and their bounds, one sequence at a time."""
    k, d = w.shape
    b, n = x.shape[:2]
    W, B = w.double(), bias.double() if bias is not None else torch.zeros(d).double().cuda()
    y, s1, ey = (torch.zeros(b, m, d, dtype=torch.float64, device="cuda") for m in (n, k - 1, n))
    dx, ds0, edx, eds0 = (torch.zeros_like(t) for t in (y, s1, y, s1))
    dw, db, edw, edb = (torch.zeros_like(t) for t in (W, B, W, B))
    rows = b * -(-n // 32) + 4 * 64  # of partial sums, more than there are
    for i in range(b):
        m = n if lens is None else max(0, min(n, int(lens[i])))
        past = s0[i].double() if s0 is not None else torch.zeros(k - 1, d).double().cuda()
        seq = torch.cat([past, x[i, :m].double()])
        pre, mag = B.expand(m, d).clone(), B.abs().expand(m, d).clone()
        for j in range(k):
            pre += W[j] * seq[j:j + m]
            mag += (W[j] * seq[j:j + m]).abs()
        e0 = (k + 2) * U * mag
        sig = torch.sigmoid(pre)
        s1[i] = seq[m:]
        es = (2 * pre.abs() + 8) * U
        y[i, :m] = pre * sig if silu else pre
        ey[i, :m] = 1.1 * e0 + es * (pre * sig).abs() if silu else e0
        if dy is None:
            continue
        slope = sig + pre * sig * (1 - sig) if silu else torch.ones_like(pre)
        eslope = 0.5 * e0 + (es + 4 * U) * (sig + (pre * sig).abs()) if silu else 0 * e0
        g = dy[i, :m].double()
        e, ee = g * slope, g.abs() * (eslope + U * slope.abs())
        dseq, eseq = torch.zeros_like(seq), torch.zeros_like(seq)
        if ds1 is not None:
            dseq[m:] += ds1[i].double()
        for j in range(k):
            dseq[j:j + m] += W[j] * e
            eseq[j:j + m] += W[j].abs() * (ee + (k + 2) * U * e.abs())
            dw[j] += (e * seq[j:j + m]).sum(0)
            edw[j] += ((ee + (32 + 4 + rows / 64 + 64) * U * e.abs()) * seq[j:j + m].abs()).sum(0)
        if ds1 is not None:
            eseq[m:] += U * (dseq[m:].abs() + ds1[i].double().abs())
        db += e.sum(0)
        edb += (ee + (32 + 4 + rows / 64 + 64) * U * e.abs()).sum(0)
        dx[i, :m], ds0[i] = dseq[k - 1:], dseq[:k - 1]
        edx[i, :m], eds0[i] = eseq[k - 1:], eseq[:k - 1]
    return dict(y=(y, ey), s1=(s1, 0 * s1), dx=(dx, edx), dw=(dw, edw), db=(db, edb),
                ds0=(ds0, eds0))


def check(name, got, ref):
    want, bound = ref
    close(got, want, bound + (half_step(got.dtype, want) if got.dtype != F32 else 0), name)


CASES = [  # b, l, d, taps, lengths, bias, state, act
    (1, 1, 1, 1, None, True, False, "silu"), (1, 1, 8, 4, None, True, True, "silu"),
    (2, 2, 5, 4, None, False, True, "none"), (3, 5, 16, 2, None, True, False, "silu"),
    (2, 33, 24, 3, None, True, True, "silu"), (1, 130, 100, 4, None, False, False, "silu"),
    (2, 67, 65, 8, None, True, True, "none"), (2, 40, 512, 5, None, True, True, "silu"),
    (4, 70, 72, 4, [70, 0, 1, 33], True, True, "silu"), (3, 9, 7, 6, [2, 9, 0], True, True, "none"),
    (3, 40, 64, 7, [50, -3, 5], False, False, "silu"), (2, 1000, 264, 4, [1000, 997], True, True, "silu")]


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("b,l,d,k,lens,with_bias,state,act", CASES)
def test_causal_conv(b, l, d, k, lens, with_bias, state, act, dtype):
    log(f"case causal conv {b} {l} {d} {k} {lens} {with_bias} {state} {act} {dtype}")
    x, dy = randn(1, b, l, d, dtype=dtype), randn(2, b, l, d, dtype=dtype)
    w = randn(3, k, d, dtype=dtype, scale=k ** -0.5)
    bias = randn(4, d, dtype=dtype, scale=0.3) if with_bias else None
    s0 = randn(5, b, k - 1, d, dtype=dtype) if state else None
    ds1 = randn(6, b, k - 1, d, dtype=dtype) if state else None
    lengths = torch.tensor(lens, dtype=torch.int32, device="cuda") if lens else None
    ref = reference(x, w, bias, s0, lens, act == "silu", dy, ds1)
    if lens:  # nothing past a length is read
        for i, m in enumerate(lens):
            x[i, max(m, 0):], dy[i, max(m, 0):] = float("nan"), float("inf")
    y, s1 = dwc.causal_conv(x, w, bias, s0, lengths, act)
    dx, dw, db, ds0 = dwc.causal_conv_bwd(dy, ds1, x, w, bias, s0, lengths, act)
    sync()
    for name, got in (("y", y), ("s1", s1), ("dx", dx), ("dw", dw), ("db", db), ("ds0", ds0)):
        if got is not None:
            check(name, got, ref[name])
    assert (db is None) == (bias is None) and (ds0 is None) == (s0 is None)
    assert torch.equal(s1.double(), ref["s1"][0])
    ys, ss = dwc.causal_conv_step(x, w, bias, s0, lengths, act)
    assert torch.equal(ys, y) and torch.equal(ss, s1)
    again = dwc.causal_conv_bwd(dy, ds1, x, w, bias, s0, lengths, act)
    for s, t in zip(again, (dx, dw, db, ds0)):
        assert s is t is None or torch.equal(s, t)


@pytest.mark.parametrize("wt", [F32, F16])
def test_weights_of_another_type_and_strides(wt):
    """Operands inside wider tensors, aligned and not, weights in fp32."""
    b, l, d, k = 2, 37, 40, 4
    for lo in (0, 8, 3):
        big, gbig = randn(1, b, l, 96, dtype=BF16), randn(2, l, b, 96, dtype=BF16)
        x, dy = big[..., lo:lo + d], gbig.transpose(0, 1)[..., lo:lo + d]
        w, bias = randn(3, k, d, dtype=wt, scale=0.5), randn(4, d, dtype=wt)
        ref = reference(x, w, bias, None, None, True, dy, None)
        y, s1 = dwc.causal_conv(x, w, bias, act="silu")
        dx, dw, db, _ = dwc.causal_conv_bwd(dy, None, x, w, bias, act="silu")
        sync()
        for name, got in (("y", y), ("s1", s1), ("dx", dx), ("dw", dw), ("db", db)):
            check(f"{name} {lo}", got, ref[name])
        assert torch.equal(y, dwc.causal_conv(x.contiguous(), w, bias, act="silu")[0])


def test_pieces_give_the_whole():
    """Calls on consecutive pieces, whole and token by token, in place."""
    x, w = randn(1, 2, 50, 48, dtype=F16), randn(2, 4, 48, dtype=F16, scale=0.5)
    whole, end = dwc.causal_conv(x, w, act="silu")
    out, state = [], torch.zeros_like(end)
    for lo, hi in ((0, 1), (1, 3), (3, 20), (20, 21), (21, 50)):
        if hi - lo > 5:
            y, state = dwc.causal_conv(x[:, lo:hi], w, s0=state, act="silu")
        else:
            y, s1 = dwc.causal_conv_step(x[:, lo:hi], w, s0=state, act="silu", out_state=state)
            assert s1 is state
        out.append(y)
    assert torch.equal(torch.cat(out, 1), whole) and torch.equal(state, end)


def test_gradient_by_differences():
    x, w, bias = (randn(i, *s) for i, s in enumerate([(2, 6, 3), (3, 3), (3,)]))
    s0, dy, ds1 = randn(5, 2, 2, 3), randn(6, 2, 6, 3), randn(7, 2, 2, 3)
    lens = [6, 1]

    def f(x, w, bias, s0):
        r = reference(x, w, bias, s0, lens, True)
        return ((r["y"][0] * dy.double()).sum() + (r["s1"][0] * ds1.double()).sum()).item()

    got = dwc.causal_conv_bwd(dy, ds1, x, w, bias, s0,
                              torch.tensor(lens, dtype=torch.int32, device="cuda"), "silu")
    args, step = [t.double() for t in (x, w, bias, s0)], 1e-5
    for a, g in zip(args, got):
        for i in range(a.numel()):
            flat, old = a.view(-1), a.view(-1)[i].item()
            flat[i] = old + step
            up = f(*args)
            flat[i] = old - step
            down = f(*args)
            flat[i] = old
            # step^2 of the third derivative and 64-bit noise / step: < 1e-6 here
            assert abs((up - down) / (2 * step) - g.view(-1)[i].item()) < 2e-5


def test_empty_and_far():
    w = randn(1, 4, 8)
    y, s1 = dwc.causal_conv(torch.empty(0, 5, 8, device="cuda"), w)
    assert y.shape == (0, 5, 8) and s1.shape == (0, 3, 8)
    s0 = randn(2, 2, 3, 8)
    y, s1 = dwc.causal_conv(torch.empty(2, 0, 8, device="cuda"), w, s0=s0)
    assert y.shape == (2, 0, 8) and torch.equal(s1, s0)
    e = torch.empty(2, 0, 8, device="cuda")
    dx, dw, _, ds0 = dwc.causal_conv_bwd(e, s0, e, w, None, s0)
    assert (dw == 0).all() and torch.equal(ds0, s0)
    _, dw, db, _ = dwc.causal_conv_bwd(torch.empty(0, 5, 8, device="cuda"), None,
                                       torch.empty(0, 5, 8, device="cuda"), w, w[0].contiguous())
    assert (dw == 0).all() and (db == 0).all()
    # tokens more than 2^32 elements apart
    far = torch.empty_strided((1, 3, 64), (0, (1 << 31) + 64, 1), dtype=BF16, device="cuda")
    near = randn(3, 1, 3, 64, dtype=BF16)
    far.copy_(near)
    w = randn(4, 4, 64, dtype=BF16)
    assert torch.equal(dwc.causal_conv(far, w)[0], dwc.causal_conv(near, w)[0])
    for s, t in zip(dwc.causal_conv_bwd(far, None, far, w),
                    dwc.causal_conv_bwd(near, None, near, w)):
        assert s is t is None or torch.equal(s, t)


def test_values_at_the_ends_of_the_range():
    """SiLU's limits, and an infinity or NaN only where its taps reach."""
    x = torch.tensor([-200.0, 200.0, -1e30, 1e30, 0.0, 0.0, 0.0, 0.0], device="cuda")
    w = torch.tensor([[1.0]], device="cuda")
    y, _ = dwc.causal_conv(x.view(1, -1, 1), w, act="silu")
    assert torch.equal(y.flatten()[[1, 3]], x[[1, 3]]) and (y.flatten()[[0, 2, 4]] == 0).all()
    x = randn(1, 1, 40, 16)
    x[0, 20, 3] = float("inf")
    y, _ = dwc.causal_conv(x, randn(2, 4, 16).abs() + 0.1)
    bad = ~torch.isfinite(y[0])
    assert bad.sum() == 4 and bad[20:24, 3].all()


def test_refusals():
    x, w = randn(1, 2, 5, 8), randn(2, 4, 8)
    z = torch.zeros(2, 3, 8, device="cuda")
    for bad, args, kw in [
            (ValueError, (x[0], w), {}), (ValueError, (x, w[0]), {}),
            (ValueError, (x, w.t().contiguous()), {}), (ValueError, (x, w.t()), {}),
            (ValueError, (x.transpose(1, 2), randn(3, 4, 5)), {}),
            (TypeError, (x, w, w[0].half()), {}), (TypeError, (x.half(), w, None, z), {}),
            (ValueError, (x, w, None, z[:, :2]), {}), (ValueError, (x, w), dict(act="relu")),
            (ValueError, (x, w), dict(lengths=torch.zeros(3, dtype=torch.int32, device="cuda"))),
            (TypeError, (x, w), dict(lengths=torch.zeros(2, dtype=torch.int64, device="cuda"))),
            (dwc.DwcError, (x, randn(4, 9, 8)), {})]:
        with pytest.raises(bad):
            dwc.causal_conv(*args, **kw)
    with pytest.raises(ValueError):
        dwc.causal_conv_step(x, w, s0=z, out_state=z[:1])
    with pytest.raises(dwc.DwcError):  # y would be written over its input's state
        dwc.causal_conv_step(x, w, s0=z, out_state=x.view(-1)[:48].view(2, 3, 8))
    with pytest.raises(ValueError):
        dwc.causal_conv_bwd(x[:, :4], None, x, w)
