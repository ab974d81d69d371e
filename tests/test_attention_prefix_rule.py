"""When a shared prefix has a pass of its own: where rereading it costs, and not for prompts, whose rows fill row tiles by
themselves and only pay for the partial results.  Seen in the workspace, which then holds parts of the prefix.  Runs without a
GPU."""
import os

import pytest

from conftest import ROOT

LIB = os.path.join(ROOT, "weight_only_quantized_w4a16_amd", "libqgemm.so")
pytestmark = pytest.mark.skipif(not os.path.exists(LIB), reason="libqgemm.so not built")


def passes(B, n, prefix, G=4, Hkv=8, D=128, known=True):
    from weight_only_quantized_w4a16_amd import ops
    size = lambda shared: ops.paged_attention_workspace_bytes(B * n, B, prefix // 64 + 20, G * Hkv, Hkv, D, 64, shared, n if known else 0)
    return size(prefix) != size(0)


@pytest.mark.parametrize("known", [True, False])
def test_prompts_have_none(known):
    for B, n, G in ((16, 32, 4), (32, 256, 4), (8, 512, 4), (4, 128, 1), (64, 64, 8)):
        assert not passes(B, n, 8192, G, known=known), (B, n, G)


@pytest.mark.parametrize("known", [True, False])
def test_decode_steps_and_proposals_have_one(known):
    for B, n, G in ((16, 1, 4), (32, 8, 4), (128, 1, 8), (16, 31, 4), (64, 4, 4)):
        assert passes(B, n, 8192, G, known=known), (B, n, G)
    for B, prefix in ((4, 512), (2, 8192), (1, 16384)):      # little to reread
        assert not passes(B, 1, prefix, known=known), (B, prefix)
