"""The selective scan in chunks, each case with the form that the host's
workspace says it takes: two blocks of states, chunks of 32 to 128 tokens, and
more chunks than one round of the sums between them holds (128 with eight
waves, 16 with one), forward and back."""

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

from gpu_helpers import dwc, log, sync  # noqa: E402
from test_sequence_gpu import BF16, F32, randn  # noqa: E402
from test_scan_gpu import NAMES, check, inputs, reference, run_case  # noqa: E402
from test_space_cpu import scan, scan_need  # noqa: E402


def chunks(b, l, d, n, g=1):
    """How many the forward call makes of a sequence; 1 in one pass."""
    st, need = scan_need(scan(b=b, l=l, d=d, n=n, g=g), 0)
    assert st == 0
    up = lambda k: (k * 4 + 255) // 256 * 256  # noqa: E731
    lines = b * g * ((l + 31) // 32 * 32)

    def base(spl):  # A, and B and C
        np = (n + spl - 1) // spl * spl
        return up(np * d) + up(lines * 2 * np), np

    if need == base(16)[0]:
        return 1
    rest, np = base(4 if n <= 4 else (8 if n <= 8 else 16))
    for nc in range(2, (l + 31) // 32 + 1):
        if need == rest + up(b * nc * np * d) + up(b * nc * d):
            return nc
    raise AssertionError("a workspace of another layout")


@pytest.mark.parametrize("b,l,d,n,g,nc,lens", [
    # two and three blocks of 16 states
    (2, 700, 9, 17, 3, 22, [1, 700]), (1, 600, 12, 32, 1, 19, None), (1, 650, 70, 45, 1, 21, [633]),
    # chunks of 88 and of 128 tokens
    (200, 700, 2, 65, 1, 8, None), (820, 300, 2, 65, 1, 3, None),
    # more than 128 chunks: eight waves take two rounds
    (1, 4200, 10, 3, 1, 132, None), (2, 4400, 5, 20, 1, 138, [4400, 4097]),
    # more than 16: one wave takes two, back (twice) and both ways
    (256, 520, 3, 16, 1, 1, None), (52, 520, 3, 70, 1, 17, None)])
def test_rounds(b, l, d, n, g, nc, lens):
    log(f"case scan in {nc} chunks: {b} {l} {d} {n} {g}")
    assert chunks(b, l, d, n, g) == nc
    if lens is None and b > 2:
        lens = [l - (13 * i) % l for i in range(b)]
    run_case(b, l, d, n, g, lens, True, True, True, BF16)


def test_a_state_reaches_the_last_chunk():
    """Over 132 chunks, decays so near 1 that what the first state and the last
    gradient hold is most of the result."""
    b, l, d, n = 1, 4200, 70, 4
    assert chunks(b, l, d, n) == 132
    a = inputs(50, b, l, d, n, 1, F32)
    a[2] *= 1e-4
    a[3] *= 1e-3
    a[8] *= 10.0
    dy, ds1 = 1e-3 * randn(51, b, l, d), 10.0 * randn(52, b, d, n)
    ref = reference(a, None, True, dy, ds1)
    got = dwc.selective_scan(*a, softplus=True)
    got += dwc.selective_scan_bwd(dy, ds1, *a, softplus=True)
    sync()
    for name, t in zip(NAMES, got):
        check(name, t, ref[name])
