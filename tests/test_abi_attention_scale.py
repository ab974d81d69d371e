"""paged_attention refuses a scale whose base-2 form is not a finite fp32 number.
Runs without a GPU: every call fails validation, so the pointers are never dereferenced."""
import os

import pytest

from conftest import ROOT

LIB = os.path.join(ROOT, "weight_only_quantized_w4a16_amd", "libqgemm.so")
QG_OK, QG_ERR_NULL, QG_ERR_SHAPE = range(3)
FAKE = 0x4000000
ATTEND = dict(q=FAKE, k=FAKE, v=FAKE, ks=FAKE, vs=FAKE, pages=20, page=16, offsets=FAKE, len=FAKE, table=FAKE, T=4, B=2, width=4096,
              Hq=8, Hkv=2, D=128, scale=0.1, window=0, sinks=0, shared=0, max_q=0, out=FAKE, lse=FAKE, ws=None, bytes=0)

pytestmark = pytest.mark.skipif(not os.path.exists(LIB), reason="libqgemm.so not built")


@pytest.fixture(scope="module")
def attend():
    from weight_only_quantized_w4a16_amd import ops
    # keys of 4096 pages are split: without a workspace a call that passes all other checks is refused for that
    return lambda **changed: ops._lib.paged_attention(*dict(ATTEND, **changed).values(), None)


def test_scale_limits(attend):
    # scale log2(e) overflows above 3.40282e38 / 1.442695 = 2.35865e38
    for scale in (2.3588e38, -2.3588e38, 3.4e38, -3.4e38, float("inf"), float("nan")):
        assert attend(scale=scale) == QG_ERR_SHAPE, scale
    for scale in (2.3584e38, -2.3584e38, 0.0, -0.0, 1e-45, -1.0):
        assert attend(scale=scale) == QG_ERR_NULL, scale
