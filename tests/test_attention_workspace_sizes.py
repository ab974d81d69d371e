"""The workspace of paged_attention holds no parts of row tiles that no sequence can have.  Runs without a GPU."""
import os

import pytest

from conftest import ROOT

LIB = os.path.join(ROOT, "weight_only_quantized_w4a16_amd", "libqgemm.so")
pytestmark = pytest.mark.skipif(not os.path.exists(LIB), reason="libqgemm.so not built")


@pytest.mark.parametrize("B,T", [(128, 128), (256, 256), (256, 700), (1000, 1000)])
@pytest.mark.parametrize("G,Hkv,D", [(4, 8, 128), (1, 8, 64), (8, 4, 128)])
def test_ragged_batch_behind_a_shared_prefix(B, T, G, Hkv, D):
    """With max_q unknown a batch may hold long sequences and short ones.  Sequences of up to 16 rows go to the kernel that
    takes 16 rows at a time; of the others, with 17 rows or more, there are at most T G / 17, and a row tile of 128 rows for
    each of them and for every 128 rows is the most that the other kernel can need."""
    from weight_only_quantized_w4a16_amd import ops
    page, prefix, width = 64, 8192, 140
    assert (B - 1) * prefix * Hkv * D * 4 >= 64 << 20        # the prefix has a pass of its own
    need = ops.paged_attention_workspace_bytes(T, B, width, G * Hkv, Hkv, D, page, prefix, 0)
    known = ops.paged_attention_workspace_bytes(T, B, width, G * Hkv, Hkv, D, page, prefix, 1)      # no row tiles, but for G > 16
    rows = T * G
    row_tiles = rows // 128 + min(B, rows // 17)
    split = 512 // Hkv                                       # chunks that a few row tiles are split into, at most
    part = Hkv * 128 * (D + 2) * 4                           # of a row tile, all key heads
    assert need <= known + (row_tiles + split) * part


def test_a_smaller_call_may_need_more():
    """The sizes are not monotone: a workspace is for the largest size of the calls to come, not for the largest call, and one
    that is too small is refused before anything is launched."""
    from weight_only_quantized_w4a16_amd import ops
    size = lambda T, B, max_q: ops.paged_attention_workspace_bytes(T, B, 128, 32, 8, 128, 64, 0, max_q)
    assert size(8192, 1, 8192) == 0 and size(1, 1, 1) > 0
    assert size(512, 1, 512) > size(8192, 1, 8192)
    fake = 0x4000000
    call = lambda ws, n: ops._lib.paged_attention(fake, fake, fake, None, None, 200, 64, fake, fake, fake, 1, 1, 128, 32, 8, 128, 0.1, 0, 0,
                                                  0, 1, fake, None, ws, n, None)
    assert call(None, 0) == 1 and call(fake, size(1, 1, 1) - 1) == 4     # QG_ERR_NULL, QG_ERR_WORKSPACE
