"""rms_norm and swiglu with bf16, e4m3 and int8 outputs against the fp64 oracle.

Every output is the rounding of an fp32 result whose relative error is bounded
by DELTA, so it has to lie between the roundings of the fp64 value times
(1 - DELTA) and (1 + DELTA): at most one choice away, and only next to a border.

DELTA = 2^-20 (16 fp32 roundings of 2^-24).  rms_norm: x + residual 1, the
reciprocal root 1 (its sum is fp64), two products 2, the code's quotient 2.
swiglu: the hardware's 2^t 2, 1 + e 1, reciprocal 2, two products 2, the code's
quotient 2.  The exponent t = -g log2 e is off by |t| (2^-24 + 2^-26) (its
rounding, the constant's), which times ln 2 is a relative error of e of at most
|g| 2^-23 and reaches the result as e / (1 + e) of that: less than 2^-24 for
g >= 0, and |g| 2^-23 for g < 0.  Below -87 the reciprocal may vanish, an
absolute error of 2^-126 |g u|.
FLOOR = 2^-148 (two subnormal steps) bounds the absolute error of subnormal
results.
"""
import numpy as np
import pytest
import torch

from gpu_helpers import announce, dev_bf16, host_bits16
from oracle import block
from oracle import fp8_e4m3 as f8
from oracle.bf16 import bf16_bits_to_f32, f32_to_bf16_bits
from weight_only_quantized_w4a16_amd import synth

pytestmark = pytest.mark.gpu

DELTA = 2.0 ** -20
FLOOR = 2.0 ** -148
EPS = 1e-5
QMAX = {"e4m3": 448.0, "int8": 127.0}


@pytest.fixture(scope="module")
def ops():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    from weight_only_quantized_w4a16_amd import ops as _ops
    return _ops


def f64(bits):
    return bf16_bits_to_f32(bits).astype(np.float64)


def rows(M, K, seed, special=True):
    """N(0, 1) rows with a few large channels; then a zero row, rows near both ends of the range."""
    f = bf16_bits_to_f32(synth.normal_bf16((M, K), seed)).copy()
    f[:, ::7] *= 8
    rng = np.random.default_rng(seed)
    if special:
        for j, scale in enumerate([0.0, 1e30, 1e-33, 1e-39]):
            if 1 + j < M:
                f[1 + j] = rng.standard_normal(K).astype(np.float32) * np.float32(scale)
    return f32_to_bf16_bits(f)


def guarded(shape, dtype):
    """An output buffer followed by 256 guard bytes; returns (buffer, check)."""
    n = int(np.prod(shape)) * torch.empty(0, dtype=dtype).element_size()
    raw = torch.full((n + 256,), 0x5A, dtype=torch.uint8, device="cuda:0")

    def check():
        assert bool((raw[n:] == 0x5A).all()), "written past the end"
    return raw[:n].view(dtype).reshape(shape), check


def assert_bf16(y, ref, what, floor=FLOOR):
    got = f64(host_bits16(y))
    err = np.abs(ref) * DELTA + floor
    with np.errstate(over="ignore"):
        lo = f64(f32_to_bf16_bits((ref - err).astype(np.float32)))
        hi = f64(f32_to_bf16_bits((ref + err).astype(np.float32)))
    bad = ~((got >= lo) & (got <= hi))
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} values, first {np.argwhere(bad)[0]}"


def assert_codes(q, s, ref, fmt, what, floor=FLOOR):
    """Scales within DELTA of max|y| / q_max, codes the roundings of y / s."""
    s = s.cpu().numpy().astype(np.float64)
    want = np.abs(ref).max(axis=1) / QMAX[fmt]
    floor = np.broadcast_to(floor, ref.shape)
    top = np.abs(ref).max(axis=1) * DELTA + floor.max(axis=1)
    assert (np.abs(s - want) <= top / QMAX[fmt] + 2.0 ** -149).all(), f"{what}: scales"
    live = s > 0
    codes = q.cpu().numpy()
    assert not codes[~live].any(), f"{what}: codes of a zero row"
    t = ref[live] / s[live][:, None]
    err = np.abs(t) * DELTA + floor[live] / s[live][:, None]
    if fmt == "e4m3":
        got = f8.e4m3_decode(codes.view(np.uint8)[live]).astype(np.float64)
        lo = f8.e4m3_decode(f8.e4m3_encode((t - err).astype(np.float32))).astype(np.float64)
        hi = f8.e4m3_decode(f8.e4m3_encode((t + err).astype(np.float32))).astype(np.float64)
    else:
        got = codes[live].astype(np.float64)
        lo = np.clip(np.rint(t - err), -127, 127)
        hi = np.clip(np.rint(t + err), -127, 127)
    bad = ~((got >= lo) & (got <= hi))
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} codes, first {np.argwhere(bad)[0]}"


# every launch: parts of a wave (K <= 256), a wave a row (K <= 1024, or 2048 when many), 256 to 1024 threads a row, the long kernel (K > 32768)
NORM_SHAPES = [(1, 8), (5, 64), (70, 8), (37, 72), (41, 128), (19, 136), (9, 256), (6, 264), (7, 512), (6, 520), (9, 1024), (5, 1032), (1, 2048), (6, 2056), (1, 4096), (5, 4104),
               (6, 8192), (3, 8200), (5, 16384), (2, 16392), (5, 32768), (5, 32776), (2, 65536), (300, 768), (1100, 1536), (1030, 2048)]


@pytest.mark.parametrize("M,K", NORM_SHAPES)
@pytest.mark.parametrize("residual", [False, True])
def test_rms_norm(ops, M, K, residual):
    announce(f"rms_norm M={M} K={K} residual={residual}")
    x, w = rows(M, K, 1), synth.normal_bf16((K,), 3)
    r = rows(M, K, 2, special=False) if residual else None
    if residual:
        r[1:] = np.where(np.arange(M)[1:, None] % 2 == 1, r[1:], np.uint16(0))   # rows that stay at the range's ends
        if M > 6:
            r[6] = x[6] ^ np.uint16(0x8000)                                        # h = 0 exactly
    h64, y64 = block.rms_norm(f64(x), f64(r) if residual else None, f64(w), EPS)
    dx, dw = dev_bf16(x), dev_bf16(w)
    dr = dev_bf16(r) if residual else None
    what = f"M={M} K={K}"
    y, check_y = guarded((M, K), torch.bfloat16)
    h, check_h = guarded((M, K), torch.bfloat16)
    ops.rms_norm(dx, dr, dw, EPS, M, K, h, y)
    torch.cuda.synchronize()
    check_y(), check_h()
    assert_bf16(y, y64, what)
    h32 = bf16_bits_to_f32(x) if r is None else bf16_bits_to_f32(x) + bf16_bits_to_f32(r)
    hb, want = host_bits16(h), f32_to_bf16_bits(h32)
    assert np.array_equal(hb, want)
    for fmt, call, dtype in (("e4m3", ops.rms_norm_quant, torch.uint8), ("int8", ops.rms_norm_quant_int8, torch.int8)):
        q, check_q = guarded((M, K), dtype)
        s, check_s = guarded((M,), torch.float32)
        y2, check_y2 = guarded((M, K), torch.bfloat16)
        h.zero_()
        call(dx, dr, dw, EPS, M, K, h, y2, q, s)
        torch.cuda.synchronize()
        check_q(), check_s(), check_y2(), check_h()
        assert torch.equal(y2.view(torch.int16), y.view(torch.int16)) and np.array_equal(host_bits16(h), want)
        assert_codes(q, s, y64, fmt, f"{what} {fmt}")
        # without the optional outputs: the same codes
        q3, s3 = torch.empty_like(q), torch.empty_like(s)
        call(dx, dr, dw, EPS, M, K, None, None, q3, s3)
        torch.cuda.synchronize()
        assert torch.equal(q3, q) and torch.equal(s3, s)


@pytest.mark.parametrize("K", [1000, 4096, 32776])
@pytest.mark.parametrize("into", ["x", "residual"])
def test_rms_norm_in_place(ops, K, into):
    """h may overwrite x or the residual: the same bits."""
    M = 5
    announce(f"rms_norm in place K={K} into={into}")
    x, r, w = (dev_bf16(rows(M, K, s, special=False)) for s in (1, 2, 3))
    w = w[0].contiguous()
    h, y = torch.empty_like(x), torch.empty_like(x)
    q, s = torch.empty((M, K), dtype=torch.uint8, device="cuda:0"), torch.empty(M, device="cuda:0")
    ops.rms_norm_quant(x, r, w, EPS, M, K, h, y, q, s)
    q2, s2, y2 = torch.empty_like(q), torch.empty_like(s), torch.empty_like(y)
    x2, r2 = x.clone(), r.clone()
    ops.rms_norm_quant(x2, r2, w, EPS, M, K, x2 if into == "x" else r2, y2, q2, s2)
    torch.cuda.synchronize()
    assert torch.equal(x2 if into == "x" else r2, h) and torch.equal(y2, y)
    assert torch.equal(q2, q) and torch.equal(s2, s)


def test_rms_norm_eps_range(ops):
    """The smallest and a large eps."""
    M, K = 3, 256
    x, w = rows(M, K, 5), synth.normal_bf16((K,), 3)
    for eps in (np.float32(1.2e-38), np.float32(1e-6), np.float32(10.0)):
        announce(f"rms_norm eps={eps}")
        y = torch.empty((M, K), dtype=torch.bfloat16, device="cuda:0")
        ops.rms_norm(dev_bf16(x), None, dev_bf16(w), float(eps), M, K, None, y)
        torch.cuda.synchronize()
        assert_bf16(y, block.rms_norm(f64(x), None, f64(w), float(eps))[1], f"eps={eps}")


def test_rms_norm_rows_do_not_depend_on_each_other(ops):
    """A row's result is the same alone, in a batch, and beside rows of NaN."""
    M, K = 9, 4096
    announce("rms_norm row independence")
    x, w = dev_bf16(rows(M, K, 1, special=False)), dev_bf16(synth.normal_bf16((K,), 3))
    norm = ops.RMSNorm(w, EPS)
    q, s, _, y = norm.quantized(x, with_bf16=True)
    x2 = x.clone()
    x2[::2] = float("nan")
    q2, s2, _, y2 = norm.quantized(x2, with_bf16=True)
    q3, s3, _, y3 = norm.quantized(x[3:4].contiguous(), with_bf16=True)
    torch.cuda.synchronize()
    assert torch.equal(q2[1::2], q[1::2]) and torch.equal(s2[1::2], s[1::2]) and torch.equal(y2[1::2], y[1::2])
    assert torch.equal(q3[0], q[3]) and torch.equal(s3[0], s[3]) and torch.equal(y3[0], y[3])


SWIGLU_SHAPES = [(1, 8), (5, 64), (70, 8), (37, 72), (41, 128), (19, 136), (9, 256), (6, 264), (7, 512), (6, 520), (9, 1024), (5, 1032), (3, 2048), (6, 2056), (1, 4096), (4, 4104),
                 (6, 8192), (1, 14336), (5, 16384), (2, 16392), (5, 32768), (5, 32776), (300, 768), (1100, 1536), (1030, 2048)]


@pytest.mark.parametrize("M,I", SWIGLU_SHAPES)
def test_swiglu(ops, M, I):
    announce(f"swiglu M={M} I={I}")
    f = bf16_bits_to_f32(synth.normal_bf16((M, 2 * I), 1)).copy()
    f[:, :I] *= 3
    # gates over the whole range of the exponential, both signs; zeros of both signs
    f[0, :I] = np.resize(np.concatenate([np.linspace(-256, 256, 61), [0.0, -0.0]]).astype(np.float32), I)
    if M > 2:
        f[1] = 0.0
        f[2, I:] *= 1e30
    if M > 4:
        f[3, I:] *= 1e-33
        f[4, :I] = 1e-39
    gu = f32_to_bf16_bits(f)
    y64 = block.swiglu(f64(gu))
    gate, up = f64(gu)[:, :I], np.abs(f64(gu)[:, I:])
    floor = FLOOR + np.where(gate < -87, 2.0 ** -126 * -gate * up, np.maximum(-gate, 0) * 2.0 ** -23 * np.abs(y64))
    what = f"M={M} I={I}"
    d = dev_bf16(gu)
    y, check_y = guarded((M, I), torch.bfloat16)
    ops.swiglu(d, M, I, y)
    torch.cuda.synchronize()
    check_y()
    assert_bf16(y, y64, what, floor)
    for fmt, call, dtype in (("e4m3", ops.swiglu_quant, torch.uint8), ("int8", ops.swiglu_quant_int8, torch.int8)):
        q, check_q = guarded((M, I), dtype)
        s, check_s = guarded((M,), torch.float32)
        call(d, M, I, q, s)
        torch.cuda.synchronize()
        check_q(), check_s()
        assert_codes(q, s, y64, fmt, f"{what} {fmt}", floor)


def test_helpers_shapes_and_types(ops):
    announce("norm helpers: refusals")
    w = torch.ones(64, dtype=torch.bfloat16, device="cuda:0")
    x = torch.ones((2, 64), dtype=torch.bfloat16, device="cuda:0")
    norm = ops.RMSNorm(w)
    with pytest.raises(ValueError):
        norm(x[:, :32].contiguous())
    with pytest.raises(ValueError):
        norm(x, residual=x[:1])
    with pytest.raises(TypeError):
        norm(x.float())
    with pytest.raises(ValueError):
        norm(torch.ones((64, 2), dtype=torch.bfloat16, device="cuda:0").t())      # not contiguous
    with pytest.raises(ValueError):
        norm.quantized(x, fmt="int4")
    with pytest.raises(ValueError):
        ops.gated_silu(x[:, :63].contiguous())
    with pytest.raises(ops.QGemmError):
        ops.gated_silu(x[:, :24].contiguous())                                     # I = 12
    with pytest.raises(ValueError):
        ops.rms_norm(x.cpu(), None, w, EPS, 2, 64, None, x)
    y, h = norm(x)
    assert h is x and y.shape == x.shape
    empty = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda:0")
    assert norm(empty)[0].shape == (0, 64) and ops.gated_silu(empty).shape == (0, 32)


def test_many_rows_past_32_bit_offsets(ops):
    """More than 2^31 elements: the last rows are right (offsets are 64-bit)."""
    M, K = 270_000, 8192
    announce(f"rms_norm M={M} K={K}")
    x = torch.zeros((M, K), dtype=torch.bfloat16, device="cuda:0")
    tail = rows(4, K, 1, special=False)
    x[-4:] = dev_bf16(tail)
    w = synth.normal_bf16((K,), 3)
    q, s, _, y = ops.RMSNorm(dev_bf16(w), EPS).quantized(x, fmt="int8", with_bf16=True)
    torch.cuda.synchronize()
    y64 = block.rms_norm(f64(tail), None, f64(w), EPS)[1]
    assert_bf16(y[-4:], y64, "last rows")
    assert_codes(q[-4:], s[-4:], y64, "int8", "last rows")
    assert not bool(s[:-4].any())
    del q, s, y
    q, s = ops.gated_silu_quantized(x)
    torch.cuda.synchronize()
    assert_codes(q[-4:], s[-4:], block.swiglu(f64(tail)), "e4m3", "last rows")
    g = ops.gated_silu(x)
    torch.cuda.synchronize()
    assert_bf16(g[-4:], block.swiglu(f64(tail)), "last rows")
