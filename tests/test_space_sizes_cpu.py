"""What the selective scan and the residual norm ask for as workspace, and
which sizes they take, without a GPU."""

import ctypes
import os

import pytest

import depthwise_convolution_dwc_amd as dwc
from test_space_cpu import norm, scan, scan_need

pytestmark = pytest.mark.skipif(not os.path.exists(dwc.LIB_PATH), reason="libdwc.so not built")


@pytest.mark.parametrize("b,l,d", [(8, 2048, 2048), (32, 6000, 4096), (300, 129, 64)])
def test_one_pass_holds_no_chunks(b, l, d):
    """A, and B and C in fp32 in lines of 32 up to whole chunks of 32 tokens."""
    a = (16 * d * 4 + 255) // 256 * 256
    assert scan_need(scan(b=b, l=l, d=d, n=16, g=1), 0) == (0, a + b * ((l + 31) // 32 * 32) * 128)


def test_chunks_hold_their_states():
    st, need = scan_need(scan(b=1, l=4096, d=256, n=16, g=1), 0)
    assert st == 0 and need >= 16 * 256 * 4 + 4096 * 128 + 4096 // 128 * 16 * 256 * 4


def test_limits_of_chunks_are_not_those_of_one_pass():
    """More sequences times channels than the chunks' launches take."""
    assert scan_need(scan(b=65535, l=129, d=2112, n=16, g=1), 0)[0] == 0


@pytest.mark.parametrize("c,resident", [(771, 1280), (1023, 1280), (1031, 768), (1500, 768),
                                        (2047, 768)])
@pytest.mark.parametrize("rows", [700, 3333, 16384])
def test_odd_rows_of_the_norm_are_spread_over_resident_workgroups(rows, c, resident):
    """Five waves a SIMD hold four values a lane, three hold eight; a workgroup
    leaves a row of three partial sums."""
    need = ctypes.c_size_t()
    p = norm(rows=rows, c=c, x=2, y=2)
    assert dwc.lib().dwc_residual_norm_bwd_workspace_size(ctypes.byref(p), ctypes.byref(need)) == 0
    rounds = -(-rows // resident)
    assert need.value == -(-rows // rounds) * 3 * c * 4
