"""The selective scan where decays grow: products of them past fp32's range
that meet states or gradients of zero, or small enough that the result is in
range.  Every form then gives what the definition gives token by token, to the
bounds that stand in test_scan_gpu.

Here operands of 1e-30 and 1e-25 meet, whose products are below 2^-149.  A
product that is below 2^-126 comes out as a multiple of 2^-149, off by half of
that at most; an output (dC over its channels, say) is a sum of fewer than 2^23
products, so TINY = 2^-126 >= 2^23 2^-150 more covers them all."""

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

from gpu_helpers import dwc, log, sync  # noqa: E402
from test_sequence_gpu import F32, randn  # noqa: E402
from test_scan_gpu import NAMES, TINY, check, inputs, reference  # noqa: E402


def growing(b, l, d, n, gate):
    """Half of the states grow by e^3.5 at each of the tokens 32 to 63, so by
    e^112 = 4e48 over them.  They start from zero in every other channel and
    from about 1e-25 in the rest, and nothing joins them before token 64; what
    reaches them from behind is about 1e-30."""
    a = inputs(40, b, l, d, n, 1, F32, gate=gate, soft=False)
    u, delta, A, s0 = a[0], a[1], a[2], a[8]
    delta *= 0.01
    delta[:, 32:64] = 3.5
    u[:, :64] = 0.0
    A[:, ::2] = 1.0
    s0[:, ::2, ::2] = 0.0
    s0[:, 1::2, ::2] *= 1e-25
    dy, ds1 = randn(41, b, l, d), randn(42, b, d, n)
    dy[:, 32:] *= 1e-30
    ds1 *= 1e-30
    return a, dy, ds1


def run(a, dy, ds1, lengths):
    got = dwc.selective_scan(*a, lengths=lengths)
    got += dwc.selective_scan_bwd(dy, ds1, *a, lengths=lengths)
    got += dwc.selective_scan_step(*a, lengths=lengths)
    sync()
    return got


# one pass; chunks of 8, 4 and 16 states a lane; several blocks of states; one
# wave over all chunks
@pytest.mark.parametrize("b,l,d,n,lens,gate", [
    (2, 150, 70, 16, [150, 77], True), (1, 600, 20, 5, None, True), (1, 500, 10, 3, None, False),
    (1, 600, 30, 16, [590], True), (1, 600, 9, 70, None, True), (3, 130, 66, 33, None, False),
    (300, 100, 3, 16, None, True)])
def test_growing_decays(b, l, d, n, lens, gate):
    log(f"case scan growing {b} {l} {d} {n}")
    a, dy, ds1 = growing(b, l, d, n, gate)
    lengths = torch.tensor(lens, dtype=torch.int32, device="cuda") if lens else None
    ref = reference(a, lens, False, dy, ds1)
    assert all(torch.isfinite(ref[k][0]).all() for k in NAMES if ref[k][0] is not None)
    got = run(a, dy, ds1, lengths)
    for name, t in zip(NAMES + ("y", "s1"), got):
        if t is not None:
            check(name, t, (ref[name][0], ref[name][1] + TINY))
    # steps below zero with the signs of A and B turned too: the same numbers
    a[1], a[2], a[3] = -a[1], -a[2], -a[3]
    for name, s, t in zip(NAMES + ("y", "s1"), got, run(a, dy, ds1, lengths)):
        if s is not None:
            assert torch.equal(s, -t if name in ("ddelta", "dA", "dB") else t), name
