"""The largest sizes that the gated unit accepts fit one launch.

Runs without a GPU: refused calls reach no launch.
"""
import os

import pytest

from conftest import ROOT

LIB = os.path.join(ROOT, "weight_only_quantized_w4a16_amd", "libqgemm.so")
QG_ERR_SHAPE = 2
FAKE = 0x4000000

pytestmark = pytest.mark.skipif(not os.path.exists(LIB), reason="libqgemm.so not built")


def test_elements_past_a_launch_are_refused():
    """One thread handles eight elements, 256 threads a workgroup, and a launch holds fewer than 2^32 threads: from
    2^35 - 2047 elements on, the gated unit's last workgroup would be the one too many."""
    from weight_only_quantized_w4a16_amd import ops
    M, I = 65537, 524280
    assert 2 ** 35 - 2048 < M * I < 2 ** 35 and I % 8 == 0
    assert ops._lib.swiglu(FAKE, M, I, FAKE, None) == QG_ERR_SHAPE
