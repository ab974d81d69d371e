"""kv_append into an 8-bit cache: the codes and scales of every value head are those that quant_act_per_token gives its D
elements (IEEE fp32 quotients, rounded to the nearest code), bit for bit, and so are those of keys that are neither normed
nor rotated."""
import numpy as np
import pytest
import torch

from gpu_helpers import announce
from oracle import fp8_e4m3 as f8

pytestmark = pytest.mark.gpu


def heads_of(kind, T, H, D, rng):
    """[T, H, D] bf16: ordinary values; magnitudes over many binades; values of few digits, whose quotients meet ties; scales
    about 2^-100, below which rows divide, and subnormal ones."""
    x = rng.standard_normal((T, H, D))
    if kind == "wide":
        x *= np.exp2(rng.integers(-12, 13, (T, H, D)))
    elif kind == "few digits":
        x = rng.integers(-28, 29, (T, H, D)) * np.exp2(rng.integers(-3, 1, (T, H, D)))
    elif kind == "small":
        x *= np.exp2(rng.integers(-125, -85, (T, H, 1)).astype(float))
    return torch.from_numpy(x).to(torch.bfloat16)


@pytest.mark.parametrize("kind", ["normal", "wide", "few digits", "small"])
@pytest.mark.parametrize("D", [64, 128])
def test_codes_of_heads(kind, D):
    from weight_only_quantized_w4a16_amd import ops
    rng = np.random.default_rng(D)
    Hq, Hkv, page, T = 4, 4, 64, 2000
    pages = (T + page - 1) // page
    k, v = heads_of(kind, T, Hkv, D, rng), heads_of(kind, T, Hkv, D, rng)
    qkv = torch.cat((torch.zeros((T, Hq, D), dtype=torch.bfloat16), k, v), 1).reshape(T, -1).contiguous().cuda()
    cache = ops.PagedKVCache(pages, Hkv, D, page, "e4m3")
    table = torch.from_numpy(rng.permutation(pages).astype(np.int32))
    announce(f"codes of heads, {kind}, D={D}")
    ops.PagedAttention(cache, Hq).append(qkv, table.view(1, -1).cuda(), torch.tensor([0, T], dtype=torch.int32, device="cuda"),
                                         torch.tensor([T], dtype=torch.int32, device="cuda"))
    at = torch.arange(T)
    page_of, slot = table[at // page].long(), at % page
    for name, x in (("k", k), ("v", v)):
        codes = getattr(cache, name).cpu()[page_of, :, slot]
        scales = getattr(cache, name + "_scale").cpu()[page_of, :, slot]
        f = x.float().numpy()
        s = (np.abs(f).max(-1) / np.float32(448)).astype(np.float32)
        assert np.array_equal(scales.numpy(), s), name
        with np.errstate(all="ignore"):
            quotient = np.where(s[..., None] > 0, f / s[..., None], np.float32(0))
        # (a zero row has codes 0)
        want = np.where(s[..., None] > 0, f8.e4m3_encode(np.clip(quotient, -448, 448).astype(np.float32)), 0)
        differ = codes.numpy() != want
        assert not differ.any(), f"{name}: {differ.sum()} codes of {differ.size}, {differ.any(-1).sum()} rows"
        if D == 128:
            M = T * Hkv
            q, sa = torch.empty((M, D), dtype=torch.uint8, device="cuda"), torch.empty(M, dtype=torch.float32, device="cuda")
            ops.quant_act_per_token(x.reshape(M, D).contiguous().cuda(), M, D, q, sa)
            assert torch.equal(q.cpu().reshape(codes.shape), codes) and torch.equal(sa.cpu().reshape(scales.shape), scales), name
