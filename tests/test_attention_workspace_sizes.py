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
