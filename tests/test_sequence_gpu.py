"""Layer norm, dropout and the token form of the gated delta rule against
plain formulations in 64 bits.

Bounds.  u = 2^-24 and half = finfo(t).eps / 2 for an output of type t.  A
sum in these kernels runs over at most 32 values in a lane, then a tree of
at most 10 levels: under 64 roundings a value's path, so a sum is off by at
most 64 u times the sum of its terms' magnitudes (Higham, Accuracy and
Stability of Numerical Algorithms, chapter 3).
"""

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

from gpu_helpers import dwc, log, sync  # noqa: E402

U = 2.0 ** -24
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16


def half(t):
    return torch.finfo(t).eps / 2


def half_step(t, want):
    """Half a step of type t at the values ``want``: below the smallest
    normal number steps stop shrinking (2^-24 for float16)."""
    return half(t) * want.abs().clamp_min(torch.finfo(t).tiny)


def randn(seed, *shape, dtype=F32, scale=1.0, shift=0.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g, dtype=torch.float64) * scale + shift).to(dtype).cuda()


def close(got, want, bound, what):
    g = got.double()
    assert g.shape == want.shape, what
    worst = ((g - want).abs() / (bound + 1e-300)).max().item() if g.numel() else 0.0
    log(f"{what}: {worst:.3g} of the bound")
    assert torch.isfinite(g).all(), what
    assert worst <= 1.0, (what, worst)


# ------------------------------------------------------------- layer norm ----

NORM = [(rows, c, x, y) for rows, c in
        [(1, 1), (3, 2), (5, 8), (33, 24), (49, 64), (7, 100), (130, 257), (65, 512), (17, 1000),
         (9, 1031), (5, 2048), (6, 4096), (3, 5003), (4, 8192), (2, 8193), (2, 16384), (1, 40000)]
        for x, y in [(F32, F32), (BF16, BF16), (F32, BF16), (F16, F32)]]


@pytest.mark.parametrize("rows,c,xt,yt", NORM)
def test_layer_norm(rows, c, xt, yt):
    log(f"case layer norm {rows} {c} {xt} {yt}")
    x = randn(1, rows, c, dtype=xt, scale=1.5, shift=0.7)
    w, b, dy = randn(2, c, shift=1.0), randn(3, c), randn(4, rows, c, dtype=yt)
    eps = 1e-5
    y, mean, rstd = dwc.layer_norm(x, w, b, eps=eps, out_dtype=yt)
    dx, dw, db = dwc.layer_norm_bwd(dy, x, mean, rstd, w)
    sync()
    X, W, B, DY = x.double(), w.double(), b.double(), dy.double()
    m = X.mean(1, keepdim=True)
    r = 1 / torch.sqrt(((X - m) ** 2).mean(1, keepdim=True) + eps)
    h = (X - m) * r
    # a difference is off by 64 u of the magnitudes that went into it, and
    # the norm by twice that
    H = (X.abs() + X.abs().mean(1, keepdim=True)) * r
    spread = 1 + (X.abs().mean(1, keepdim=True) * r) * U * 64  # of r, by the mean's error
    close(mean, m[:, 0], 64 * U * X.abs().mean(1), "mean")
    close(rstd, r[:, 0], 128 * U * (r * spread)[:, 0], "rstd")
    close(y, h * W + B, half_step(yt, h * W + B) + 128 * U * (H * W.abs() + B.abs()), "y")
    e = DY * W
    want = r * (e - e.mean(1, keepdim=True) - h * (e * h).mean(1, keepdim=True))
    E = e.abs() + e.abs().mean(1, keepdim=True) + H * (e.abs() * H).mean(1, keepdim=True)
    close(dx, want, half_step(xt, want) + 512 * U * r * E, "dx")
    # a column's sum: at most rows / groups terms in a lane (under 256 here),
    # 32 row groups and 64 more of the tree over workgroups
    n = min(rows, 256) + 128
    close(dw, (DY * h).sum(0), (n + 256) * U * (DY.abs() * H).sum(0), "dw")
    close(db, DY.sum(0), n * U * DY.abs().sum(0), "db")


def test_layer_norm_by_differences():
    """The gradient against central differences of the 64-bit formula."""
    x, w, b, dy = randn(5, 3, 20), randn(6, 20, shift=1.0), randn(7, 20), randn(8, 3, 20)

    def f(x, w, b):
        m = x.mean(1, keepdim=True)
        h = (x - m) / torch.sqrt(((x - m) ** 2).mean(1, keepdim=True) + 1e-5)
        return ((h * w + b) * dy.double()).sum().item()

    y, mean, rstd = dwc.layer_norm(x, w, b)
    got = dwc.layer_norm_bwd(dy, x, mean, rstd, w)
    args = [t.double() for t in (x, w, b)]
    step = 1e-5
    for a, g in zip(args, got):
        for i in range(0, a.numel(), 7):
            flat, old = a.view(-1), a.view(-1)[i].item()
            flat[i] = old + step
            up = f(*args)
            flat[i] = old - step
            down = f(*args)
            flat[i] = old
            # step^2 of the third derivative and 64-bit noise / step: < 1e-6
            # at these magnitudes; the fp32 gradient is off by far less
            assert abs((up - down) / (2 * step) - g.view(-1)[i].item()) < 2e-5


def test_layer_norm_strides_types_and_options():
    big = randn(9, 12, 80, dtype=BF16)
    x = big[:, 16:48]  # rows 80 apart, 16-byte aligned
    y, mean, rstd = dwc.layer_norm(x)
    y2, _, _ = dwc.layer_norm(x.contiguous())
    assert torch.equal(y, y2)
    x = big[:, 3:35]  # not aligned
    y, mean, rstd = dwc.layer_norm(x)
    y2, m2, r2 = dwc.layer_norm(x.contiguous())
    sync()
    want = torch.nn.functional.layer_norm(x.double(), (32,))
    close(y, want, half_step(BF16, want) + 256 * U * (1 + x.double().abs() / x.double().std()),
          "unaligned")
    dy = randn(10, 12, 80, dtype=BF16)[:, 1:33]
    a = dwc.layer_norm_bwd(dy, x, mean, rstd)
    b = dwc.layer_norm_bwd(dy.contiguous(), x.contiguous(), m2, r2)
    for s, t in zip(a, b):
        assert (s.double() - t.double()).abs().max() <= 2 * half(s.dtype) * t.double().abs().max()
    # 16-bit weights, higher rank
    x4 = randn(11, 2, 3, 5, 64, dtype=F16)
    w16, b16 = randn(12, 64, dtype=F16), randn(13, 64, dtype=F16)
    y, mean, rstd = dwc.layer_norm(x4, w16, b16)
    assert y.shape == x4.shape and mean.shape == x4.shape[:-1]
    want = torch.nn.functional.layer_norm(x4.double(), (64,), w16.double(), b16.double())
    close(y, want, half_step(F16, want) + 128 * U * 16, "16-bit weights")
    out = torch.empty_like(x4)
    y2, _, _ = dwc.layer_norm(x4, w16, b16, out=out)
    assert y2 is out and torch.equal(out, y)


def test_layer_norm_no_rows_constant_rows_and_non_finite_rows():
    x = torch.empty(0, 16, device="cuda")
    y, mean, rstd = dwc.layer_norm(x)
    dx, dw, db = dwc.layer_norm_bwd(x, x, mean, rstd)
    assert y.shape == (0, 16) and not dw.any() and not db.any()
    x = torch.full((2, 300), 3.25, device="cuda")
    y, mean, rstd = dwc.layer_norm(x, eps=1e-5)
    assert not y.any() and torch.equal(mean, torch.full_like(mean, 3.25))
    x = randn(14, 4, 64)
    ref = dwc.layer_norm(x)[0]
    x[1, 5], x[2, 7] = float("nan"), float("inf")
    y = dwc.layer_norm(x)[0]
    assert torch.equal(y[0], ref[0]) and torch.equal(y[3], ref[3])
    assert y[1].isnan().all() and y[2].isnan().all()


def test_layer_norm_large_mean():
    """A mean 1000 times the spread: the two-pass form keeps the spread."""
    x = randn(15, 8, 1024, shift=1000.0)
    y, mean, rstd = dwc.layer_norm(x)
    X = x.double()
    want = torch.nn.functional.layer_norm(X, (1024,), eps=1e-5)
    H = 2 * X.abs() / X.std(1, keepdim=True)
    close(y, want, 128 * U * H, "large mean")


def test_layer_norm_same_bits_and_refusals():
    x, dy = randn(16, 3000, 320, dtype=BF16), randn(17, 3000, 320, dtype=BF16)
    y, mean, rstd = dwc.layer_norm(x)
    a, b = (dwc.layer_norm_bwd(dy, x, mean, rstd) for _ in range(2))
    for s, t in zip(a, b):
        assert torch.equal(s, t)
    with pytest.raises(ValueError):
        dwc.layer_norm(x.t())  # last axis not dense
    with pytest.raises(ValueError):
        dwc.layer_norm(x, torch.ones(319, device="cuda"))
    with pytest.raises(TypeError):
        dwc.layer_norm(x, torch.ones(320, device="cuda"), torch.ones(320, device="cuda").half())
    with pytest.raises(TypeError):
        dwc.layer_norm(x.double())
    with pytest.raises(dwc.DwcError):
        dwc.layer_norm(x, eps=-1.0)
    with pytest.raises(ValueError):
        dwc.layer_norm_bwd(dy[:5], x, mean, rstd)
    with pytest.raises(ValueError):
        dwc.layer_norm(x.float().expand(3000, 320)[:1].expand(4, 320))  # rows overlap


# ---------------------------------------------------------------- dropout ----

def philox_kept(n, p, seed, offset):
    """The definition in numpy's 64-bit integers."""
    u, m = np.uint64, np.uint64(0xFFFFFFFF)
    with np.errstate(over="ignore"):
        at = np.arange((n + 3) // 4, dtype=u) + u(offset)
        c = [at & m, at >> u(32), np.zeros_like(at), np.zeros_like(at)]
        k = [seed & 0xFFFFFFFF, seed >> 32]
        for _ in range(7):
            a, b = c[0] * u(0xD2511F53), c[2] * u(0xCD9E8D57)
            c = [(b >> u(32)) ^ c[1] ^ u(k[0]), b & m, (a >> u(32)) ^ c[3] ^ u(k[1]), a & m]
            k = [(k[0] + 0x9E3779B9) % (1 << 32), (k[1] + 0xBB67AE85) % (1 << 32)]
    return torch.from_numpy(np.stack(c, 1).reshape(-1)[:n] >= u(round(p * 2 ** 32))).cuda()


@pytest.mark.parametrize("dt", [F32, BF16, F16])
@pytest.mark.parametrize("n", [1, 2, 3, 5, 8, 1000, 4099, 65537])
@pytest.mark.parametrize("p,seed,offset", [(0.1, 1, 0), (0.5, (1 << 63) + 77, (1 << 32) - 3),
                                           (0.25, (1 << 64) - 1, (1 << 64) - 5)])
def test_dropout(dt, n, p, seed, offset):
    log(f"case dropout {dt} {n} {p} {seed} {offset}")
    x, r = randn(n, n, dtype=dt), randn(n + 1, n, dtype=dt)
    kept = philox_kept(n, p, seed, offset)
    for res in (None, r):
        y = dwc.dropout(x, p, seed, offset, residual=res)
        sync()
        v = torch.where(kept, x.double() / (1 - p), 0.0)
        want = v if res is None else v + res.double()
        # the scale, the product and the sum each round once in fp32
        mag = v.abs() + (0 if res is None else res.double().abs())
        close(y, want, half_step(dt, want) + 4 * U * mag, "dropout")
        if res is None:
            assert torch.equal(y != 0, kept & (x != 0))


def test_dropout_edges():
    x = randn(1, 4000)
    assert torch.equal(dwc.dropout(x, 0.0, 5), x)
    assert not dwc.dropout(x, 1.0, 5).any()
    assert torch.equal(dwc.dropout(x, 1.0, 5, residual=x), x)
    kept = philox_kept(4000, 0.5, 9, 0)
    bad = torch.where(kept, x, float("nan"))
    assert torch.equal(dwc.dropout(bad, 0.5, 9), dwc.dropout(x, 0.5, 9))  # dropped NaN: 0
    y = dwc.dropout(x[1:], 0.5, 9)  # an address that no wide load takes
    assert torch.equal(y, dwc.dropout(x[1:].clone(), 0.5, 9))
    assert dwc.dropout(x[:0], 0.5, 9).shape == (0,)
    # the second half of a tensor, from the offset where it begins
    assert torch.equal(dwc.dropout(x, 0.5, 9, 3)[2000:], dwc.dropout(x[2000:], 0.5, 9, 503))
    for args in ((-0.1, 1), (1.5, 1), (float("nan"), 1)):
        with pytest.raises(dwc.DwcError):
            dwc.dropout(x, *args)
    for args in ((0.5, -1), (0.5, 1 << 64), (0.5, 1, -1)):
        with pytest.raises(ValueError):
            dwc.dropout(x, *args)
    with pytest.raises(ValueError):
        dwc.dropout(x.view(40, 100).t(), 0.5, 1)
    with pytest.raises(TypeError):
        dwc.dropout(x, 0.5, 1, residual=x.half())


def test_dropout_share_kept():
    n, p = 1 << 22, 0.3
    y = dwc.dropout(torch.ones(n, device="cuda"), p, 1234)
    share = (y != 0).double().mean().item()
    assert abs(share - (1 - p)) < 6 * (p * (1 - p) / n) ** 0.5  # six deviations


# ------------------------------------------- gated delta rule, token by token ----

def delta_inputs(seed, b, n, hk, hv, dk, dv, dtype, state=True):
    mixed = torch.empty(b, n, 2 * hk * dk + hv * dv + 3, dtype=dtype, device="cuda")
    qk = randn(seed, b, n, 2 * hk, dk)
    mixed[..., :2 * hk * dk] = (qk / qk.norm(dim=-1, keepdim=True)).flatten(2).to(dtype)
    mixed[..., 2 * hk * dk:] = randn(seed + 1, b, n, hv * dv + 3).to(dtype)
    q = mixed[..., :hk * dk].unflatten(-1, (hk, dk))
    k = mixed[..., hk * dk:2 * hk * dk].unflatten(-1, (hk, dk))
    v = mixed[..., 2 * hk * dk:2 * hk * dk + hv * dv].unflatten(-1, (hv, dv))
    g = -0.3 * torch.nn.functional.softplus(randn(seed + 2, b, n, hv))
    beta = torch.sigmoid(randn(seed + 3, b, n, hv))
    s0 = randn(seed + 4, b, hv, dk, dv, scale=0.3) if state else None
    return q, k, v, g, beta, s0


def delta_reference(q, k, v, g, beta, s0, lengths=None, scale=None):
    """Token by token in 64 bits, and the magnitudes that each output sums."""
    b, n, hv, dv = v.shape
    hk, dk = q.shape[2:]
    scale = dk ** -0.5 if scale is None else scale
    q, k = (t.double().repeat_interleave(hv // hk, 2) for t in (q, k))
    v, a, beta = v.double(), g.double().exp(), beta.double()
    s = torch.zeros(b, hv, dk, dv, dtype=torch.float64, device=v.device) if s0 is None \
        else s0.double()
    o = torch.zeros_like(v)
    for t in range(n):
        dec = s * a[:, t, :, None, None]
        u = beta[:, t, :, None] * (v[:, t] - (dec * k[:, t, :, :, None]).sum(2))
        new = dec + k[:, t, :, :, None] * u[:, :, None, :]
        ot = scale * (new * q[:, t, :, :, None]).sum(2)
        if lengths is not None:
            live = (t < lengths)[:, None, None]
            new = torch.where(live[..., None], new, s)
            ot = torch.where(live, ot, 0.0)
        s, o[:, t] = new, ot
    return o, s


def rel(got, want):
    d, w = (got.double() - want).norm().item(), want.norm().item()
    return d / w if w else d


# An update's roundings: at most 64 u of what it sums, which the contraction
# of the rule (|a| <= 1, |1 - beta k k^T| <= 1 for |k| = 1, beta in 0..1)
# does not grow; over the tokens that a state remembers (some tens at these
# decays) the norm stays under 1e-5.
S_TOL = 1e-5


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("b,n,hk,hv,dk,dv", [
    (1, 1, 1, 1, 1, 1), (1, 1, 8, 8, 128, 128), (3, 1, 2, 6, 96, 72), (2, 4, 1, 2, 100, 75),
    (5, 1, 2, 2, 33, 7), (2, 3, 1, 1, 256, 40), (1, 9, 3, 3, 64, 64), (2, 1, 1, 3, 20, 130)])
def test_delta_step(dtype, b, n, hk, hv, dk, dv):
    log(f"case delta step {dtype} {b, n, hk, hv, dk, dv}")
    for state in (True, False):
        a = delta_inputs(b + n, b, n, hk, hv, dk, dv, dtype, state)
        o, s1 = dwc.delta_rule_step(*a)
        sync()
        wo, ws = delta_reference(*a)
        assert rel(s1, ws) < S_TOL
        assert rel(o, wo) < half(dtype) + S_TOL


def test_delta_step_in_place_lengths_and_masked_places():
    a = list(delta_inputs(3, 4, 3, 2, 4, 64, 32, BF16))
    lengths = torch.tensor([0, 1, 3, 2], dtype=torch.int32, device="cuda")
    wo, ws = delta_reference(*a, lengths=lengths)
    for t in a[:3]:  # what stands past a sequence's end is not used
        for i, n in enumerate(lengths.tolist()):
            t[i, n:] = float("nan")
    a[3], a[4] = a[3].clone(), a[4].clone()
    for i, n in enumerate(lengths.tolist()):
        a[3][i, n:], a[4][i, n:] = float("inf"), float("nan")
    s = a[5].clone()
    o, s1 = dwc.delta_rule_step(*a[:5], s, lengths=lengths, out_state=s)
    sync()
    assert s1 is s and torch.equal(s[0], a[5][0]) and not o[0].any()
    assert rel(s, ws) < S_TOL and rel(o, wo) < half(BF16) + S_TOL


def test_delta_step_forgets_and_refuses():
    q, k, v, g, beta, s0 = delta_inputs(4, 2, 1, 2, 2, 32, 16, F32)
    o, s1 = dwc.delta_rule_step(q, k, v, torch.full_like(g, -float("inf")), beta, s0)
    wo, ws = delta_reference(q, k, v, g, beta, None)
    assert rel(s1, ws) < S_TOL and rel(o, wo) < S_TOL
    assert torch.isfinite(s1).all()
    with pytest.raises(ValueError):
        dwc.delta_rule_step(q, k, v, g[:, :, :1], beta, s0)
    with pytest.raises(ValueError):
        dwc.delta_rule_step(q, k[..., :16], v, g, beta, s0)
    with pytest.raises(TypeError):
        dwc.delta_rule_step(q, k, v.half(), g, beta, s0)
    with pytest.raises(TypeError):
        dwc.delta_rule_step(q, k, v, g, beta.half(), s0)
    with pytest.raises(ValueError):
        dwc.delta_rule_step(q, k, v, g, beta, s0.transpose(2, 3))
    with pytest.raises(ValueError):
        dwc.delta_rule_step(q.expand(2, 1, 2, 32)[..., ::2], k[..., ::2], v, g, beta, s0)


def test_another_stream():
    """Operands made on one stream, the calls on another."""
    side = torch.cuda.Stream()
    x = randn(20, 2000, 512, dtype=BF16)
    a = delta_inputs(21, 2, 1, 2, 2, 64, 64, BF16)
    sync()
    want = dwc.layer_norm(x)[0], dwc.dropout(x, 0.5, 3), dwc.delta_rule_step(*a)[1]
    sync()
    side.wait_stream(torch.cuda.current_stream())
    got = (dwc.layer_norm(x, stream=side)[0], dwc.dropout(x, 0.5, 3, stream=side),
           dwc.delta_rule_step(*a, stream=side.cuda_stream)[1])
    side.synchronize()
    for s, t in zip(got, want):
        assert torch.equal(s, t)
