"""What the selective scan asks for as workspace, and which sizes it takes,
without a GPU."""

import os

import pytest

import depthwise_convolution_dwc_amd as dwc
from test_space_cpu import scan, scan_need

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
