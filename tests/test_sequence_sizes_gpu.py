"""The sequence layer's operators where their kernels take other paths than
at small odd sizes: many rows, many heads, operands whose addresses and
strides allow wide loads.  References and bounds are those of
test_sequence_gpu.py and test_delta_gpu.py."""

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import test_delta_gpu as delta  # noqa: E402
import test_sequence_gpu as base  # noqa: E402
from gpu_helpers import dwc, log, sync  # noqa: E402
from test_sequence_gpu import BF16, F16, F32, S_TOL, delta_inputs, half, rel  # noqa: E402


def aligned(a):
    """q, k and v as tensors of their own."""
    return [t.contiguous() for t in a[:3]] + list(a[3:])


# more rows than one step of the backward pass takes, an odd number past it
@pytest.mark.parametrize("rows,c", [(9001, 8), (4099, 24), (5003, 100), (4097, 512), (2051, 1031),
                                    (1025, 2048), (515, 8192), (259, 9001)])
@pytest.mark.parametrize("xt,yt", [(F32, F32), (BF16, BF16), (F16, F32)])
def test_layer_norm_many_rows(rows, c, xt, yt):
    base.test_layer_norm(rows, c, xt, yt)


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("b,n,hk,hv,dk,dv", [
    (1, 2, 2, 4, 64, 64), (2, 1, 1, 1, 200, 12),            # two lanes across
    (33, 1, 4, 8, 100, 75), (9, 3, 8, 16, 128, 132),        # eight lanes across
    (40, 1, 8, 8, 24, 64), (17, 2, 4, 16, 60, 64), (20, 1, 8, 8, 256, 128)])
def test_delta_step_many_heads(dtype, b, n, hk, hv, dk, dv):
    log(f"case delta step {dtype} {b, n, hk, hv, dk, dv}")
    a = delta_inputs(b + dk, b, n, hk, hv, dk, dv, dtype)
    lengths = torch.arange(b, dtype=torch.int32, device="cuda") % (n + 1)
    for x in (a, aligned(a)):
        for m in (None, lengths):
            o, s1 = dwc.delta_rule_step(*x, lengths=m)
            sync()
            wo, ws = base.delta_reference(*x, lengths=m)
            assert rel(s1, ws) < S_TOL
            assert rel(o, wo) < half(dtype) + S_TOL


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("shape", [(2, 130, 2, 2, 128, 128), (1, 200, 1, 1, 64, 72),
                                   (2, 100, 2, 4, 96, 40), (1, 64, 1, 5, 128, 64),
                                   (1, 65, 2, 2, 56, 196)])
def test_delta_chunked_wide_loads(dtype, shape):
    log(f"case delta wide {dtype} {shape}")
    delta.check(aligned(delta_inputs(sum(shape), *shape, dtype)))


# column blocks past 512, an odd number of them a head
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("shape", [(4, 70, 16, 32, 100, 75), (3, 130, 32, 64, 64, 48),
                                   (5, 66, 32, 32, 40, 130), (2, 64, 32, 64, 128, 128)])
def test_delta_chunked_many_heads(dtype, shape):
    log(f"case delta many heads {dtype} {shape}")
    a = delta_inputs(sum(shape), *shape, dtype)
    delta.check(a)
    lengths = (torch.arange(shape[0], dtype=torch.int32, device="cuda") * 37) % (shape[1] + 1)
    delta.check(aligned(a), lengths)
