"""Codes of rows whose scale is subnormal: a quotient past the largest code is
saturated to it, with its sign.

A scale s = max|y| / q_max below 2^-126 is a whole number of steps of 2^-149, so
y / s may exceed q_max by far more than roundings: max|y| = 178 steps gives an
int8 scale of one step and a quotient of 178.  The rows here hold y = n 2^-149
exactly, with n up to 20000:

* gated unit: gate 2^-70 (its sigmoid rounds to 1/2), up n 2^-78;
* norm: h = (1, n 2^-34, ...) in 2^2j columns, the weight 0 for the first and
  2^(-115 - j) for the others: the mean of h^2 is 2^-2j (1 + d), d < 2^-34, so
  the reciprocal root is 2^j to a last bit and n stays whole to a thousandth.

The scale is then the IEEE quotient of n_max 2^-149 by q_max, and a code is the
rounding of y / s to one unit in the quotient's last place, clamped.
"""
import numpy as np
import pytest
import torch

from gpu_helpers import announce, dev_bf16
from oracle import fp8_e4m3 as f8
from oracle.bf16 import f32_to_bf16_bits

pytestmark = pytest.mark.gpu

QMAX = {"e4m3": 448.0, "int8": 127.0}
STEP = np.float32(2.0 ** -149)
# largest n of a row: around the borders of one to a few scale steps in both formats, all with 8 bits of mantissa
TOPS = [1, 63, 64, 100, 127, 178, 190, 191, 223, 225, 250, 300, 400, 448, 472, 600, 656, 672, 1112, 2432, 5024, 20096]


@pytest.fixture(scope="module")
def ops():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    from weight_only_quantized_w4a16_amd import ops as _ops
    return _ops


def values(K, seed):
    """Whole numbers [len(TOPS), K] with 8 bits of mantissa, row i's largest TOPS[i] at both signs."""
    rng = np.random.default_rng(seed)
    n = np.zeros((len(TOPS), K))
    for i, top in enumerate(TOPS):
        v = np.floor(rng.random(min(K, 66) - 3) * top)
        v = np.minimum(np.where(v >= 256, np.floor(v / 128) * 128, v), top)
        n[i, 1:1 + v.size] = v * rng.choice([-1.0, 1.0], v.size)
        n[i, 1 + v.size], n[i, 2 + v.size] = top, -top
        n[i, 1:] = rng.permutation(n[i, 1:])
    return n


def check(q, s, n, fmt, what):
    y = n.astype(np.float32) * STEP
    want_s = np.abs(y).max(axis=1) / np.float32(QMAX[fmt])
    got_s = s.cpu().numpy()
    assert np.array_equal(got_s, want_s), f"{what}: scales"
    codes = q.cpu().numpy()
    assert not codes[want_s == 0].any(), f"{what}: codes of a zero scale"
    live = want_s > 0
    t = (y[live] / want_s[live][:, None]).astype(np.float64)
    lo, hi = t - np.abs(t) * 2.0 ** -23, t + np.abs(t) * 2.0 ** -23
    if fmt == "e4m3":
        dec = lambda c: f8.e4m3_decode(c).astype(np.float64)
        got = dec(codes.view(np.uint8)[live])
        lo, hi = (dec(f8.e4m3_encode(np.clip(v, -448, 448).astype(np.float32))) for v in (lo, hi))
    else:
        got = codes[live].astype(np.float64)
        lo, hi = (np.clip(np.rint(v), -127, 127) for v in (lo, hi))
    bad = ~((got >= lo) & (got <= hi))
    rows = [TOPS[i] for i in np.nonzero(live)[0]]
    assert not bad.any(), f"{what}: {bad.sum()} codes, first in the row of largest {rows[np.argwhere(bad)[0][0]]}"


CALLS = {"e4m3": ("_quant", torch.uint8), "int8": ("_quant_int8", torch.int8)}


# parts of a wave, a wave, workgroups, the long kernel
@pytest.mark.parametrize("I", [64, 256, 512, 2048, 14336, 32776])
@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_swiglu(ops, I, fmt):
    announce(f"saturated codes swiglu I={I} {fmt}")
    n = values(I, I)
    M = n.shape[0]
    gu = np.concatenate([np.full((M, I), 2.0 ** -70), n * 2.0 ** -78], axis=1).astype(np.float32)
    name, dtype = CALLS[fmt]
    q, s = torch.empty((M, I), dtype=dtype, device="cuda:0"), torch.empty(M, device="cuda:0")
    getattr(ops, "swiglu" + name)(dev_bf16(f32_to_bf16_bits(gu)), M, I, q, s)
    torch.cuda.synchronize()
    check(q, s, n, fmt, f"I={I} {fmt}")


@pytest.mark.parametrize("K", [64, 256, 1024, 4096, 16384, 65536])
@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_rms_norm(ops, K, fmt):
    announce(f"saturated codes norm K={K} {fmt}")
    n = values(K, K)
    M = n.shape[0]
    j = int(np.log2(K)) // 2
    assert 4 ** j == K
    x = (n * 2.0 ** -34).astype(np.float32)
    x[:, 0] = 1.0
    w = np.full(K, 2.0 ** (-149 + 34 - j), np.float32)
    w[0] = 0.0
    eps = float(np.finfo(np.float32).tiny)
    d_x, d_w = dev_bf16(f32_to_bf16_bits(x)), dev_bf16(f32_to_bf16_bits(w))
    name, dtype = CALLS[fmt]
    q, s = torch.empty((M, K), dtype=dtype, device="cuda:0"), torch.empty(M, device="cuda:0")
    getattr(ops, "rms_norm" + name)(d_x, None, d_w, eps, M, K, None, None, q, s)
    torch.cuda.synchronize()
    check(q, s, n, fmt, f"K={K} {fmt}")
