"""The short causal convolution at sizes where a lane takes strips of 16 and 32
tokens, whose loops then run several times with their loads ahead, with lengths
that end inside a strip, at its end and up to the taps past it.  Bounds as in
test_conv_gpu."""

import ctypes

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

from gpu_helpers import dwc, log, sync  # noqa: E402
from test_sequence_gpu import BF16, F16, F32, randn  # noqa: E402
from test_conv_gpu import check, reference  # noqa: E402
from test_space_cpu import conv  # noqa: E402


def strips_of(b, l, d, k):
    """Strips of a sequence in the backward pass, up to the next four: each four
    leave a row of partial sums."""
    need = ctypes.c_size_t()
    assert dwc.lib().dwc_causal_conv_bwd_workspace_size(ctypes.byref(conv(b=b, l=l, d=d, k=k)),
                                                        ctypes.byref(need)) == 0
    return need.value // (b * (k + 1) * d * 4) * 4


def up4(n):
    return -(-n // 4) * 4


@pytest.mark.parametrize("b,l,d,k,strip,dtype,lens", [
    (8, 515, 4096, 4, 32, BF16, None), (8, 515, 4096, 8, 32, F16, [515, 512, 513, 480, 481, 39, 7, 0]),
    (8, 515, 4099, 4, 32, F16, [515, 514, 512, 510, 65, 64, 63, 1]), (8, 515, 4099, 8, 32, F32, None),
    (16, 270, 4096, 1, 32, F32, None), (64, 97, 2048, 2, 32, BF16, [97 - i % 70 for i in range(64)]),
    (8, 300, 4096, 7, 16, BF16, [300, 288, 289, 294, 272, 16, 17, 15]),
    (8, 301, 4098, 3, 16, F32, [301, 300, 288, 290, 289, 33, 18, 2]), (8, 257, 4100, 6, 16, F16, None),
    (8, 257, 4098, 5, 16, BF16, None)])
@pytest.mark.parametrize("state", [True, False])
def test_strips(b, l, d, k, strip, dtype, lens, state):
    log(f"case causal conv in strips of {strip}: {b} {l} {d} {k} {lens} {dtype} {state}")
    assert strips_of(b, l, d, k) == up4(-(-l // strip))
    act = "silu" if state or k % 2 else "none"
    x, dy = randn(1, b, l, d, dtype=dtype), randn(2, b, l, d, dtype=dtype)
    w = randn(3, k, d, dtype=dtype, scale=k ** -0.5)
    bias = randn(4, d, dtype=dtype, scale=0.3) if state else None
    s0 = randn(5, b, k - 1, d, dtype=dtype) if state else None
    ds1 = randn(6, b, k - 1, d, dtype=dtype) if state else None
    lengths = torch.tensor(lens, dtype=torch.int32, device="cuda") if lens else None
    ref = reference(x, w, bias, s0, lens, act == "silu", dy, ds1)
    if lens:  # nothing past a length is read
        for i, m in enumerate(lens):
            x[i, m:], dy[i, m:] = float("nan"), float("inf")
    y, s1 = dwc.causal_conv(x, w, bias, s0, lengths, act)
    dx, dw, db, ds0 = dwc.causal_conv_bwd(dy, ds1, x, w, bias, s0, lengths, act)
    sync()
    for name, got in (("y", y), ("s1", s1), ("dx", dx), ("dw", dw), ("db", db), ("ds0", ds0)):
        if got is not None:
            check(name, got, ref[name])
    assert torch.equal(s1.double(), ref["s1"][0])
    ys, ss = dwc.causal_conv_step(x, w, bias, s0, lengths, act)
    assert torch.equal(ys, y) and torch.equal(ss, s1)
    for s, t in zip(dwc.causal_conv_bwd(dy, ds1, x, w, bias, s0, lengths, act), (dx, dw, db, ds0)):
        assert s is t is None or torch.equal(s, t)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_one_tap_in_small_strips(dtype):
    """Without tokens before a strip the loop of four runs twice in one of 8."""
    b, l, d = 2, 37, 24
    assert strips_of(b, l, d, 1) == up4(-(-l // 8))
    x, dy, w = randn(1, b, l, d, dtype=dtype), randn(2, b, l, d, dtype=dtype), randn(3, 1, d)
    ref = reference(x, w, None, None, [37, 20], True, dy)
    lengths = torch.tensor([37, 20], dtype=torch.int32, device="cuda")
    y, s1 = dwc.causal_conv(x, w, lengths=lengths, act="silu")
    dx, dw, db, ds0 = dwc.causal_conv_bwd(dy, None, x, w, lengths=lengths, act="silu")
    assert s1.shape == (b, 0, d) and db is None and ds0 is None
    for name, got in (("y", y), ("dx", dx), ("dw", dw)):
        check(name, got, ref[name])
