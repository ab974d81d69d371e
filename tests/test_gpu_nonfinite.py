"""Values that overflowed or went wrong further up stay visible: an activation or
a coded output never turns them into ordinary numbers.

Finite inputs reach all of these: a product's fp32 accumulators overflow, and so
do x + residual and silu(gate) * up.
"""
import numpy as np
import pytest
import torch

from gpu_helpers import announce, dev_bf16, host_bits16
from oracle import int4_g128 as q4
from oracle.bf16 import bf16_bits_to_f32, f32_to_bf16_bits

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ops():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    from weight_only_quantized_w4a16_amd import ops as _ops
    return _ops


# a decode kernel of one and of several waves a tile, its K split, the small-M
# kernel of one, two and four row tiles, the large one with and without a K split
PRODUCTS = [(3, 8256, 1024), (1, 256, 4096), (16, 1024, 14336), (9, 528, 1280), (17, 512, 512), (40, 1040, 1024),
            (100, 4096, 4096), (130, 14336, 256), (520, 14336, 256)]


def overflowing(ops, M, N, K, act):
    """(y, kind): rows of kind 0 add 1.4e37 to a bias of +-3.38e38, rows of kind 1 subtract it; even columns have the
    positive bias.  In rows of kind 2 two groups' fp32 sums overflow with opposite signs."""
    codes = np.full((K, N), 8, np.uint8)                             # zero weights but in the first two groups
    codes[:128], codes[128:256] = 15, 1                              # 7 and -7 times the scale
    scales = np.full((K // 128, N), f32_to_bf16_bits(np.float32(2e36)), np.uint16)
    packed, scales = q4.pack_native(codes, scales)
    w = ops.Int4G128Weight(torch.from_numpy(packed.view(np.int32)).cuda(), torch.from_numpy(scales.view(np.int16)).cuda(), K, N)
    kind = np.arange(M) % 3 if M > 2 else np.full(M, 2)
    a = np.zeros((M, K), np.float32)
    a[kind == 0, 5] = 1.0
    a[kind == 1, 200] = 1.0
    a[kind == 2, 5] = a[kind == 2, 200] = 3e38
    bias = np.where(np.arange(N) % 2 == 0, 3.38e38, -3.38e38).astype(np.float32)
    y = ops.W4A16Linear(w, dev_bf16(f32_to_bf16_bits(bias)), act)(dev_bf16(f32_to_bf16_bits(a)))
    torch.cuda.synchronize()
    return bf16_bits_to_f32(host_bits16(y)), kind


@pytest.mark.parametrize("M,N,K", PRODUCTS)
def test_relu_keeps_nan(ops, M, N, K):
    announce(f"relu of nan M={M} N={N} K={K} {ops.w4a16_kernel_for(M, N, K)}")
    y, kind = overflowing(ops, M, N, K, "relu")
    assert np.isnan(y[kind == 2]).all()
    assert np.isposinf(y[kind == 0][:, ::2]).all() and not y[kind == 0][:, 1::2].any()
    assert not y[kind == 1][:, 1::2].any() and np.isfinite(y[kind == 1][:, ::2]).all()


@pytest.mark.parametrize("M,N,K", PRODUCTS)
@pytest.mark.parametrize("act", ["gelu", "gelu_tanh", "silu"])
def test_activations_of_infinity(ops, M, N, K, act):
    """act(+inf) = +inf, act(nan) = nan; far below zero the result is a zero (at -inf: nan, infinity times zero)."""
    announce(f"{act} of infinity M={M} N={N} K={K}")
    y, kind = overflowing(ops, M, N, K, act)
    assert np.isnan(y[kind == 2]).all()
    assert np.isposinf(y[kind == 0][:, ::2]).all() and not y[kind == 0][:, 1::2].any()
    assert np.isfinite(y[kind == 1][:, ::2]).all() and not np.nan_to_num(y[kind == 1][:, 1::2]).any()


FORMATS = {"e4m3": ("_quant", torch.uint8), "int8": ("_quant_int8", torch.int8)}
# parts of a wave, a wave, workgroups, the long kernel; more rows: one wave a row up to 2048 columns
ROWS = [(6, 8), (6, 72), (6, 256), (6, 512), (6, 1024), (6, 2056), (6, 14336), (6, 32776), (1100, 1536)]


def coded(ops, op, fmt, *args):
    M, K = args[-2:]
    q, s = torch.empty((M, K), dtype=FORMATS[fmt][1], device="cuda:0"), torch.empty(M, device="cuda:0")
    extra = (None, None) if op == "rms_norm" else ()
    getattr(ops, op + FORMATS[fmt][0])(*args, *extra, q, s)
    torch.cuda.synchronize()
    return q.cpu().numpy(), s.cpu().numpy()


def check_coded(got, clean, bad):
    """The scales of the rows in `bad` are no numbers or infinite; the other rows are as without them."""
    (q, s), (q0, s0) = got, clean
    good = np.setdiff1d(np.arange(s.size), bad)
    assert not np.isfinite(s[bad]).any(), s[bad]
    assert np.array_equal(q[good], q0[good]) and np.array_equal(s[good], s0[good]) and np.isfinite(s[good]).all()


@pytest.mark.parametrize("M,I", ROWS)
@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_swiglu_codes(ops, M, I, fmt):
    announce(f"swiglu codes of non-finite rows M={M} I={I} {fmt}")
    rng = np.random.default_rng(I)
    gu = rng.standard_normal((M, 2 * I)).astype(np.float32)
    clean = coded(ops, "swiglu", fmt, dev_bf16(f32_to_bf16_bits(gu)), M, I)
    c = rng.integers(0, I, 4)
    gu[0, I + c[0]] = np.nan
    gu[1, c[1]] = np.nan
    gu[3, :] = np.nan
    gu[4, c[2]] = gu[4, I + c[2]] = 3e38                             # their product overflows
    gu[5, c[3]], gu[5, I + c[3]] = np.inf, 0.0
    got = coded(ops, "swiglu", fmt, dev_bf16(f32_to_bf16_bits(gu)), M, I)
    check_coded(got, clean, np.array([0, 1, 3, 4, 5]))


@pytest.mark.parametrize("M,K", ROWS)
@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_rms_norm_codes(ops, M, K, fmt):
    announce(f"norm codes of non-finite rows M={M} K={K} {fmt}")
    rng = np.random.default_rng(K)
    x, r = (rng.standard_normal((M, K)).astype(np.float32) for _ in range(2))
    w = dev_bf16(f32_to_bf16_bits(rng.standard_normal(K).astype(np.float32)))
    run = lambda w: coded(ops, "rms_norm", fmt, *(dev_bf16(f32_to_bf16_bits(v)) for v in (x, r)), w, 1e-5, M, K)
    clean = run(w)
    c = rng.integers(0, K, 3)
    x[0, c[0]] = np.nan
    x[2, :] = np.nan
    x[3, c[1]] = r[3, c[1]] = 3e38                                   # their sum overflows
    r[5, c[2]] = -np.inf
    check_coded(run(w), clean, np.array([0, 2, 3, 5]))
    w[K // 2] = float("nan")                                         # a weight that is no number: in every row
    q, s = run(w)
    assert not np.isfinite(s).any()
