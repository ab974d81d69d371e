"""paged_attention takes the scale vectors of its cache at any 4-byte address, as kv_append does.  Runs
without a GPU: every call fails validation, so the pointers are never dereferenced."""
import os

import pytest

from conftest import ROOT

LIB = os.path.join(ROOT, "weight_only_quantized_w4a16_amd", "libqgemm.so")
QG_OK, QG_ERR_NULL, QG_ERR_SHAPE, QG_ERR_ALIGN = range(4)
FAKE = 0x4000000
ATTEND = dict(q=FAKE, k=FAKE, v=FAKE, ks=FAKE, vs=FAKE, pages=20, page=16, offsets=FAKE, len=FAKE, table=FAKE, T=4, B=2, width=4096,
              Hq=8, Hkv=2, D=128, scale=0.1, window=0, sinks=0, shared=0, max_q=0, out=FAKE, lse=FAKE, ws=None, bytes=0)

pytestmark = pytest.mark.skipif(not os.path.exists(LIB), reason="libqgemm.so not built")


@pytest.fixture(scope="module")
def attend():
    from weight_only_quantized_w4a16_amd import ops
    # keys of 4096 pages are split: without a workspace a call that passes all other checks is refused for that
    return lambda **changed: ops._lib.paged_attention(*dict(ATTEND, **changed).values(), None)


def test_alignment_of_scale_vectors(attend):
    for at in (4, 8, 12, 16):
        assert attend(ks=FAKE + at) == QG_ERR_NULL and attend(vs=FAKE + at) == QG_ERR_NULL, at
    for at in (1, 2, 6):
        assert attend(ks=FAKE + at) == QG_ERR_ALIGN and attend(vs=FAKE + at) == QG_ERR_ALIGN, at
