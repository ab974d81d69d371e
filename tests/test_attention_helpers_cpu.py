"""The attention helpers check types and shapes before any call; workspace sizes; frequencies.  Runs without a GPU."""
import os

import pytest
import torch

from conftest import ROOT

LIB = os.path.join(ROOT, "weight_only_quantized_w4a16_amd", "libqgemm.so")
pytestmark = pytest.mark.skipif(not os.path.exists(LIB), reason="libqgemm.so not built")


@pytest.fixture(scope="module")
def ops():
    from weight_only_quantized_w4a16_amd import ops as _ops
    return _ops


def test_refusals(ops):
    cache = ops.PagedKVCache(4, 2, 64, 16, "e4m3", device="cpu")
    assert cache.k.shape == (4, 2, 16, 64) and cache.k.dtype == torch.uint8 and cache.v_scale.shape == (4, 2, 16)
    plain = ops.PagedKVCache(4, 2, 64, 16, device="cpu")
    assert plain.k_scale is None and plain.v.dtype == torch.bfloat16
    with pytest.raises(ValueError, match="fmt"):
        ops.PagedKVCache(4, 2, 64, 16, "int8", device="cpu")
    w, f = torch.ones(64, dtype=torch.bfloat16), ops.rotary_frequencies(64, device="cpu")
    with pytest.raises(TypeError, match="q_weight"):
        ops.PagedAttention(cache, 4, f, torch.ones(64))
    with pytest.raises(ValueError, match="k_weight"):
        ops.PagedAttention(cache, 4, f, w, w[:32])
    with pytest.raises(TypeError, match="inv_freq"):
        ops.PagedAttention(cache, 4, f.float())
    layer = ops.PagedAttention(cache, 4, f, w, w)
    assert layer.rotary_dim == 64 and layer.scale == 0.125
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32)
    qkv, table, offsets, kv = torch.zeros((3, 512), dtype=torch.bfloat16), i32(1, 2).view(1, 2), i32(0, 3), i32(3)
    for bad, what in (((qkv[:, :500], table, offsets, kv), "qkv"), ((qkv, table[0], offsets, kv), "block_table"),
                      ((qkv, i32(1, 2, 3, 4).view(2, 2), offsets, kv), "block_table"), ((qkv, table, kv, kv), "q_offsets")):
        with pytest.raises(ValueError, match=what):
            layer.append(*bad)
    with pytest.raises(TypeError, match="kv_len"):
        layer.append(qkv, table, offsets, kv.long())
    with pytest.raises(ValueError, match="on the GPU"):
        layer.append(qkv, table, offsets, kv)
    with pytest.raises(ValueError, match="q:"):
        layer.attend(qkv.view(3, 8, 64), table, offsets, kv)
    with pytest.raises(ValueError, match="positions"):
        ops.norm_rope(qkv, i32(0, 1), 4, 2, 64)


def test_frequencies(ops):
    f = ops.rotary_frequencies(8, 10000.0, device="cpu")
    assert f.dtype == torch.float64
    assert torch.allclose(f, torch.tensor([1.0, 0.1, 0.01, 0.001], dtype=torch.float64), rtol=1e-14, atol=0)


def test_workspace_sizes_stay_moderate(ops):
    """Partial results are those of split keys: none for a large prefill, tens of MB at most for decoding."""
    assert ops.paged_attention_workspace_bytes(8192, 1, 512, 32, 8, 128, 64, 0, 8192) == 0
    for B in (1, 4, 16, 64, 256):
        for width in (1, 8, 512, 4096):
            assert ops.paged_attention_workspace_bytes(B, B, width, 32, 8, 128, 16, 0, 1) <= 64 << 20
