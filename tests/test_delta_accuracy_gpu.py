"""What single values of the chunked gated delta rule and of its gradients are
worth: outputs of 16 bits before they are rounded, the gradient of every
decay, small magnitudes, small tokens beside large ones.  Norms of whole
outputs are tested in test_delta_gpu.py, whose F bounds an output's error
before its rounding as a share of its 2-norm.
"""

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

from gpu_helpers import dwc, log, sync  # noqa: E402
from test_delta_gpu import F, TOL, check, wanted  # noqa: E402
from test_sequence_gpu import BF16, F16, F32, delta_inputs, half, randn, rel  # noqa: E402


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("shape", [(1, 200, 2, 2, 128, 128), (2, 130, 1, 2, 64, 64),
                                   (1, 150, 2, 4, 96, 72)])
def test_16_bit_outputs_are_rounded_once(dtype, shape):
    """Against the exact values rounded to the type.  An output that is off
    by d before it is rounded comes out as the next value of its type, a step
    away, with probability d / step, so the squares sum to
    sum(d step) <= F |o| eps |o|: the 2-norms' share is sqrt(F eps)."""
    log(f"case rounded once {dtype} {shape}")
    a = delta_inputs(sum(shape), *shape, dtype)
    b, n, hk, hv, dk, dv = shape
    dout, ds1 = randn(3, b, n, hv, dv, dtype=dtype), randn(4, b, hv, dk, dv, scale=0.1)
    got = dwc.delta_rule(*a)[:1] + dwc.delta_rule_bwd(dout, ds1, *a)[:3]
    sync()
    wo, _, wg = wanted(a, dout, ds1)
    for name, g, w in zip(("o", "dq", "dk", "dv"), got, [wo] + list(wg[:3])):
        r = rel(g, w.to(dtype).double())
        log(f"{name} {r:.3g}")
        assert r < (F * torch.finfo(dtype).eps) ** 0.5, (name, r)


def decay_products(a, dout, ds1):
    """dg in 64 bits and, for each token, the 2-norms' product of what it is
    the inner product of: the decayed state and its gradient."""
    q, k, v, g, beta, s0 = (t.double() for t in a)
    n, r = v.shape[1], v.shape[2] // q.shape[2]
    q, k = q.repeat_interleave(r, 2), k.repeat_interleave(r, 2)
    outer = lambda x, y: x[..., :, None] * y[..., None, :]  # noqa: E731
    down = lambda m, x: (m * x[..., :, None]).sum(-2)  # noqa: E731
    scale, s, kept = a[0].shape[3] ** -0.5, s0, []
    for t in range(n):
        dec = s * g[:, t].exp()[..., None, None]
        s = dec + outer(k[:, t], beta[:, t, :, None] * (v[:, t] - down(dec, k[:, t])))
        kept.append(dec)
    ds, dg, size = ds1.double(), torch.zeros_like(g), torch.zeros_like(g)
    for t in reversed(range(n)):
        ds = ds + scale * outer(q[:, t], dout[:, t].double())
        ds = ds - outer(k[:, t], beta[:, t, :, None] * down(ds, k[:, t]))
        dg[:, t] = (kept[t] * ds).sum((-1, -2))
        size[:, t] = kept[t].flatten(-2).norm(dim=-1) * ds.flatten(-2).norm(dim=-1)
        ds = ds * g[:, t].exp()[..., None, None]
    return dg, size


DECAYS = [(-3.0, None), (-10.0, None), (-16.0, None), (-30.0, None), (-5.0, 70), (-16.0, 70),
          (-30.0, 63), (-30.0, 64), (-60.0, 5), (-float("inf"), 70), (-float("inf"), 64)]


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("shape", [(1, 130, 2, 2, 64, 64), (1, 150, 1, 2, 128, 128),
                                   (2, 128, 1, 3, 40, 24)])
@pytest.mark.parametrize("g,at", DECAYS)
def test_gradient_of_each_decay(dtype, shape, g, at):
    """Every token's dg by itself: an inner product of the decayed state and
    its gradient, so off by at most F of their norms' product, however small
    the decay makes it.  One strong decay among mild ones, or all alike."""
    log(f"case dg {dtype} {shape} {g} {at}")
    a = list(delta_inputs(sum(shape), *shape, dtype))
    a[3] = a[3].clone()
    a[3][:, slice(None) if at is None else at] = g
    b, n, hk, hv, dk, dv = shape
    dout, ds1 = randn(5, b, n, hv, dv, dtype=dtype), randn(6, b, hv, dk, dv, scale=0.1)
    grads = dwc.delta_rule_bwd(dout, ds1, *a)
    sync()
    want, size = decay_products(a, dout, ds1)
    off = (grads[3].double() - want).abs()
    worst = (off / size.clamp_min(1e-300)).max().item()
    log(f"dg {worst:.3g}, dg of the strong one {(off / want.abs().clamp_min(1e-300))[:, at or 0].max().item():.3g}")
    assert torch.isfinite(grads[3]).all() and (off <= F * size).all(), worst
    _, _, wg = wanted(a, dout, ds1)
    for name, x, w in zip(("dq", "dk", "dv", "dg", "dbeta", "ds0"), grads, wg):
        r = rel(x, w)
        log(f"{name} {r:.3g}")
        assert r < TOL[x.dtype], (name, r)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("shape", [(1, 130, 2, 2, 64, 64), (1, 150, 1, 2, 128, 128),
                                   (2, 100, 2, 2, 40, 24)])
@pytest.mark.parametrize("power", [-80, -60, -30, 20])
def test_small_values_keep_their_bits(dtype, shape, power):
    """The gradients are linear in dout and ds1, o and s1 in v and s0: scaled
    by a power of two they come out scaled, bit by bit."""
    log(f"case small {dtype} {shape} {power}")
    a = list(delta_inputs(sum(shape), *shape, dtype))
    b, n, hk, hv, dk, dv = shape
    dout, ds1 = randn(7, b, n, hv, dv, dtype=dtype), randn(8, b, hv, dk, dv, scale=0.1)
    f = 2.0 ** power
    for name, x, y in zip(("dq", "dk", "dv", "dg", "dbeta", "ds0"),
                          dwc.delta_rule_bwd(dout * f, ds1 * f, *a),
                          dwc.delta_rule_bwd(dout, ds1, *a)):
        assert torch.equal(x, y * f), (name, rel(x, y.double() * f))
    small = a[:2] + [a[2] * f] + a[3:5] + [a[5] * f]
    for name, x, y in zip(("o", "s1"), dwc.delta_rule(*small), dwc.delta_rule(*a)):
        assert torch.equal(x, y * f), (name, rel(x, y.double() * f))
    # and for small values of everything else
    for name, x, y in zip(("dq", "dk", "dv", "dg", "dbeta", "ds0"),
                          dwc.delta_rule_bwd(dout, ds1, *small),
                          dwc.delta_rule_bwd(dout, ds1, *a)):
        assert torch.equal(x, y if name == "dv" or name == "ds0" else y * f), name


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("which", [0, 1])
def test_one_of_queries_and_keys_small_or_zero(dtype, which):
    """A product of the backward pass takes K and Q together: neither may
    cost the other its bits."""
    for f in (0.0, 2.0 ** -60, 2.0 ** 30):
        log(f"case small {dtype} {which} {f}")
        a = list(delta_inputs(9, 1, 150, 1, 2, 64, 40, dtype))
        a[which] = a[which] * f if which == 0 else a[which] * min(f, 1.0)
        check(a)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("shape", [(1, 128, 1, 2, 64, 64), (1, 150, 2, 2, 128, 128),
                                   (2, 100, 1, 2, 40, 24)])
def test_tokens_of_different_magnitudes(dtype, shape):
    """q, k, v and dout scaled by a power of two of 2^-24..1 for each token
    and checked token by token: operands have 22 bits down to 2^-17 of the
    largest of a chunk and that absolute error below it, so an output is off
    by F of its terms' size, or by F 2^-17 of the largest token's.  Terms are
    sums of up to 128 products of either sign: their size is up to 12 times
    the output's norm."""
    log(f"case magnitudes {dtype} {shape}")
    a = list(delta_inputs(sum(shape), *shape, dtype))
    b, n, hk, hv, dk, dv = shape
    dout, ds1 = randn(9, b, n, hv, dv, dtype=dtype), randn(10, b, hv, dk, dv, scale=0.1)
    gen = torch.Generator().manual_seed(11)

    def spread(t):
        return t * 2.0 ** -torch.randint(0, 25, (b, n, 1, 1), generator=gen).cuda().to(dtype)

    a[0], a[1], a[2], dout = (spread(t) for t in (a[0], a[1], a[2], dout))
    got = dwc.delta_rule(*a)[:1] + dwc.delta_rule_bwd(dout, ds1, *a)[:3]
    sync()
    wo, _, wg = wanted(a, dout, ds1)
    for name, g, w in zip(("o", "dq", "dk", "dv"), got, [wo] + list(wg[:3])):
        off, size = (g.double() - w).norm(dim=-1), w.norm(dim=-1)
        # the largest token of a head in its chunk
        top = torch.stack([size[:, t // 64 * 64:t // 64 * 64 + 64].amax(1) for t in range(n)], 1)
        bound = 12 * F * (size + 2.0 ** -17 * top) + half(g.dtype) * (g.dtype != F32) * size
        worst = (off / bound).max().item()
        log(f"{name}: {worst:.3g} of the bound")
        assert torch.isfinite(g).all() and worst <= 1.0, (name, worst)
