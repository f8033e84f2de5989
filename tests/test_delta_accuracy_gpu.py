"""What single values of the chunked gated delta rule and of its gradients are
worth: outputs of 16 bits before they are rounded.  Norms of whole outputs
are tested in test_delta_gpu.py, whose F bounds an output's error before its
rounding as a share of its 2-norm.
"""

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

from gpu_helpers import dwc, log, sync  # noqa: E402
from test_delta_gpu import F, wanted  # noqa: E402
from test_sequence_gpu import BF16, F16, F32, delta_inputs, randn, rel  # noqa: E402


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
