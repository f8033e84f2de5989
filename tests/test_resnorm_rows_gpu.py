"""The residual norm of more rows than its workgroups take at once: each walks
several sets of rows, the last one cut short, forward with the next set read
ahead and back with the columns' sums carried on.  Bounds as in
test_resnorm_gpu."""

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

from gpu_helpers import dwc, log, sync  # noqa: E402
from test_sequence_gpu import BF16, F16, F32, randn  # noqa: E402
from test_resnorm_gpu import EPS, HOW, check, reference  # noqa: E402

# Most workgroups forward: 2048, of 32 rows with 8 lanes a row down to one with
# 256; 512 with 1024 lanes; 1792 and 1024 where no wide load divides rows of
# 513 to 2048.  Half of that back, 1280 and 768 there; 64 for the columns' sums
# of rows past 8192.
SIZES = [(70001, 24), (40001, 100), (66001, 64), (18001, 257), (9001, 512), (9001, 1000),
         (4501, 2048), (5003, 771), (5003, 1031), (3001, 2047), (2500, 4096), (1100, 4100),
         (700, 5003), (1100, 8192), (131, 8200), (200, 9999)]
TYPES = [(F32, BF16), (F16, F16), (F32, F32)]


@pytest.mark.parametrize("xt,yt", TYPES)
@pytest.mark.parametrize("rows,c", SIZES)
def test_many_rows(rows, c, xt, yt):
    for act, gated, scaled, post, pre, weighted in (HOW[1], HOW[5]):
        log(f"case residual norm of many rows {rows} {c} {xt} {yt} {act}")
        x, y = randn(1, rows, c, dtype=xt), randn(2, rows, c, dtype=yt, scale=0.7)
        gate = randn(3, rows, c, dtype=yt) if gated else None
        scale = randn(4, c, shift=0.5, scale=0.3) if scaled else None
        w1, w2 = ((randn(i, c, shift=1.0, scale=0.2) for i in (5, 6)) if weighted
                  else (None, None))
        dr, dh = randn(7, rows, c, dtype=xt), randn(8, rows, c, dtype=yt) if pre else None
        kw = dict(gate=gate, scale=scale, w_post=w1, w_pre=w2, post=post, pre=pre, act=act)
        ref = reference(x, y, gate, scale, w1, w2, post, pre, act, dr, dh)
        r, h, q1, q2 = dwc.residual_norm(x, y, eps=EPS, **kw)
        grads = dwc.residual_norm_bwd(dr, dh, x, y, q1, q2, **kw)
        sync()
        for name, got in zip(("r", "h", "q1", "q2", "dx", "dy", "dgate", "dscale", "dw_post",
                              "dw_pre"), (r, h, q1, q2) + grads):
            if got is not None:
                check(name, got, ref[name])
        for s, t in zip(dwc.residual_norm_bwd(dr, dh, x, y, q1, q2, **kw), grads):
            assert s is t is None or torch.equal(s, t)
