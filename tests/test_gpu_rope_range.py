"""The head norm where x times its weight leaves fp32's range though x over its norm times the weight does not: large rows
under large weights, small rows under small ones."""
import numpy as np
import pytest
import torch

from attention_helpers import bf16
from gpu_helpers import announce
from oracle import attention as oracle
from oracle import fp8_e4m3 as f8

pytestmark = pytest.mark.gpu

EPS = 1e-30


def freqs(rot):
    return 500000.0 ** (-np.arange(rot // 2, dtype=np.float64) / max(rot // 2, 1))


# rows 2^x, weights 2^w: sums of squares at both sides of what fp32 takes, outputs within bf16's normal range
SIZES = [(48, 90), (40, 100), (30, 110), (48, -90), (-38, -100), (-30, -115), (-38, 90), (60, 80), (-60, -100), (0, 0)]


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("D,rot", [(64, 64), (128, 128), (128, 32), (64, 0)])
def test_norm_with_extreme_weights(D, rot, inter):
    from weight_only_quantized_w4a16_amd import ops
    rng = np.random.default_rng(D + rot)
    T, Hq, Hkv = 9, 6, 3
    positions = rng.integers(0, 100000, T).astype(np.int32)
    f = torch.from_numpy(freqs(rot)).cuda() if rot else None
    for ex, ew in SIZES:
        x, xt = bf16(rng.standard_normal((T, (Hq + 2 * Hkv) * D)) * 2.0 ** ex)
        w = [bf16((1 + 0.3 * rng.standard_normal(D)) * 2.0 ** ew) for _ in range(2)]
        q = torch.full((T, Hq, D), 7.0, dtype=torch.bfloat16, device="cuda")
        k = torch.full((T, Hkv, D), 7.0, dtype=torch.bfloat16, device="cuda")
        announce(f"rows 2^{ex}, weights 2^{ew}, D={D} rot={rot} inter={inter}")
        ops.qk_norm_rope(xt.cuda(), w[0][1].cuda(), w[1][1].cuda(), EPS, torch.from_numpy(positions).cuda(), f, rot, inter, T, Hq, Hkv,
                         D, q, k)
        heads = x.reshape(T, Hq + 2 * Hkv, D)
        for got, part, weight in ((q, heads[:, :Hq], w[0][0]), (k, heads[:, Hq:Hq + Hkv], w[1][0])):
            want = oracle.norm_rope(part, weight, EPS, positions, freqs(rot), rot, inter)
            # The factor (2^-23) and three products before the sum of a pair (2^-24 each), the sine and cosine (2^-22, and 2 pi
            # 2^-25 of the angle's turn): below 2^-20 of the head's largest normed value; then half a step of bf16.
            normed = np.abs(part / np.sqrt(np.mean(part * part, -1, keepdims=True) + EPS) * weight)
            near = 2.0 ** -8 * (1 + 2.0 ** -7) * np.abs(want) + 2.0 ** -20 * 2 * normed.max(-1, keepdims=True)
            with np.errstate(invalid="ignore"):
                ok = np.abs(got.double().cpu().numpy() - want) <= near
            assert ok.all(), (ex, ew, np.argwhere(~ok)[:3], got.double().cpu().numpy()[~ok][:3], want[~ok][:3])


def test_append_with_extreme_weights():
    """The same into an 8-bit cache: finite scales, and keys within a code's half step."""
    from weight_only_quantized_w4a16_amd import ops
    rng = np.random.default_rng(2)
    T, Hq, Hkv, D = 20, 2, 2, 64
    for ex, ew in SIZES:
        x, xt = bf16(rng.standard_normal((T, (Hq + 2 * Hkv) * D)) * 2.0 ** ex)
        w = bf16((1 + 0.3 * rng.standard_normal(D)) * 2.0 ** ew)
        cache = ops.PagedKVCache(2, Hkv, D, 16, "e4m3")
        layer = ops.PagedAttention(cache, Hq, torch.from_numpy(freqs(D)).cuda(), w[1].cuda(), w[1].cuda(), eps=EPS)
        i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")
        announce(f"append, rows 2^{ex}, weights 2^{ew}")
        layer.append(xt.cuda(), i32(1, 0).view(1, 2), i32(0, T), i32(T))
        part = x.reshape(T, -1, D)[:, Hq:Hq + Hkv]
        want = oracle.norm_rope(part, w[0], EPS, np.arange(T), freqs(D), D, False)
        s = cache.k_scale.double().cpu().numpy()[[1, 0]].transpose(0, 2, 1).reshape(-1, Hkv)[:T]
        c = f8.e4m3_decode(cache.k.cpu().numpy())[[1, 0]].transpose(0, 2, 1, 3).reshape(-1, Hkv, D)[:T]
        top = np.abs(want).max(-1)
        assert np.isfinite(s).all() and (np.abs(448 * s - top) <= 2.0 ** -18 * top).all(), (ex, ew)
        # half a step of a code: 2^-4 of it, 2^-10 scales of a subnormal one
        assert (np.abs(c * s[..., None] - want) <= 2.0 ** -4 * 1.01 * np.abs(want) + (2.0 ** -10 * 1.01 * s + 2.0 ** -17 * top)[..., None]).all(), (ex, ew)
