"""qgemm_w4a16_epilogue: bias, activation and residual on the product's accumulators.

The fp32 product itself comes from the plain call's kernel (same arithmetic), so
two checks pin the epilogue: every output against the fp64 oracle of the whole
formula, within half a bf16 step plus the product's own bar of 2e-2 of its RMS
times the largest slope of the activations (1.13), and, where the
product is exact (small whole numbers), within the rounding of the fp64 value:
half a bf16 step plus EPI of the terms' magnitude, the fp32 epilogue's error:
the bias sum 1 rounding of 2^-24, the activation at most 16 2^-24 relative to
max(|result|, 2^-24 |x|) plus |z| 2^-23 of its exponent (|z| <= 150 while the
exponential is above the smallest number), the residual sum 1: EPI = 2^-15.
"""
import numpy as np
import pytest
import torch

from gpu_helpers import REL_TOL, announce, dev_bf16, host_bits16
from oracle import block
from oracle import int4_g128 as q4
from oracle.bf16 import bf16_bits_to_f32, f32_to_bf16_bits
from weight_only_quantized_w4a16_amd import synth

pytestmark = pytest.mark.gpu

EPI = 2.0 ** -15


@pytest.fixture(scope="module")
def ops():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    from weight_only_quantized_w4a16_amd import ops as _ops
    return _ops


def f64(bits):
    return bf16_bits_to_f32(bits).astype(np.float64)


_W = {}


def weight(ops, K, N):
    if (K, N) not in _W:
        w = synth.weights(K, N, seed=7)
        codes, s = q4.quantize(w)
        _W[K, N] = (ops.Int4G128Weight.from_bf16(dev_bf16(w)), q4.dequant_f32(codes, s).astype(np.float64))
    return _W[K, N]


# every kernel of the product: decode (direct, several waves a tile, K split),
# small M (one, two and four row tiles), large M (each tile, K split)
SHAPES = [(1, 256, 4096), (3, 8256, 1024), (16, 8192, 2048), (4, 8192, 3968), (16, 1024, 14336), (12, 272, 16384),
          (1, 16, 128), (9, 528, 1280), (17, 512, 512), (40, 1040, 1024), (64, 4096, 8192), (65, 272, 256),
          (100, 4096, 4096), (130, 8192, 8192), (300, 2064, 384), (130, 14336, 256), (520, 14336, 256), (130, 28672, 256)]


def test_shapes_reach_every_kernel(ops):
    announce("epilogue kernels")
    names = [ops.w4a16_kernel_for(M, N, K) for M, N, K in SHAPES]
    for part in ("w4a16_decode_kernel<1,", "w4a16_decode_kernel<4,", "w4a16_small_m_kernel<1", "w4a16_small_m_kernel<2",
                 "w4a16_small_m_kernel<4", "w4a16_large_m_kernel<3, 1, 64", "w4a16_large_m_kernel<3, 1, 128",
                 "w4a16_large_m_kernel<3, 2, 64", "w4a16_large_m_kernel<3, 2, 128"):
        assert any(n.startswith(part) for n in names), (part, names)
    for kernel in ("decode", "large"):
        split = [n.rsplit("S=", 1)[1] != "1" for n in names if kernel in n]
        assert any(split) and not all(split), (kernel, names)


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_against_oracle(ops, M, N, K):
    announce(f"epilogue M={M} N={N} K={K} {ops.w4a16_kernel_for(M, N, K)}")
    wt, w64 = weight(ops, K, N)
    a = synth.activations(M, K, seed=1)
    product = f64(a) @ w64
    bias, res = synth.normal_bf16((N,), 2), synth.normal_bf16((M, N), 3)
    d_a, d_b, d_r = dev_bf16(a), dev_bf16(bias), dev_bf16(res)
    for i, act in enumerate(block.EPILOGUE_ACTIVATIONS):
        for with_bias, with_res in ((True, True), (True, False), (False, True), (False, False))[i % 2::2]:
            lin = ops.W4A16Linear(wt, d_b if with_bias else None, act)
            y = torch.full((M + 1, N), 7.0, dtype=torch.bfloat16, device="cuda:0")
            lin(d_a, out=y[:M], residual=d_r if with_res else None)
            again = lin(d_a, residual=d_r if with_res else None)
            torch.cuda.synchronize()
            assert bool((y[M] == 7.0).all())
            assert torch.equal(again, y[:M])
            ref = block.epilogue(product, f64(bias) if with_bias else None, act, f64(res) if with_res else None)
            bound = 2.0 ** -8 * (1 + 2.0 ** -8) * np.abs(ref) + 1.13 * REL_TOL * np.sqrt(np.mean(product ** 2))
            err = np.abs(f64(host_bits16(y[:M])) - ref)
            assert (err <= bound).all(), f"{act} bias={with_bias} residual={with_res}: {(err / bound).max()}"
            if with_res:                                             # the residual's own memory: the same bits
                inout = d_r.clone()
                lin(d_a, out=inout, residual=inout)
                torch.cuda.synchronize()
                assert torch.equal(inout, y[:M])


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_nothing_to_add_is_the_plain_product(ops, M, N, K):
    announce(f"epilogue none M={M} N={N} K={K}")
    wt, _ = weight(ops, K, N)
    a = dev_bf16(synth.activations(M, K, seed=1))
    lin = ops.W4A16Linear(wt)
    y = lin(a)
    ws, n = lin.workspace(M)
    z = torch.empty_like(y)
    ops.qgemm_w4a16_epilogue(a, wt.packed, wt.scales, None, "none", None, z, M, N, K, ws, n)
    # a zero bias and residual through the epilogue's own code: equal values
    zero = torch.zeros((M, N), dtype=torch.bfloat16, device="cuda:0")
    v = torch.empty_like(y)
    ops.qgemm_w4a16_epilogue(a, wt.packed, wt.scales, zero[0].contiguous(), 0, zero, v, M, N, K, ws, n)
    torch.cuda.synchronize()
    assert torch.equal(z.view(torch.int16), y.view(torch.int16)) and torch.equal(v, y)


@pytest.mark.parametrize("M", [1, 5, 16, 33, 64, 70, 200])
@pytest.mark.parametrize("act", block.EPILOGUE_ACTIVATIONS)
def test_exact_products(ops, M, act):
    """Activations of one nonzero whole number per row and weights of whole codes
    with scale 1: the product is exact, and the epilogue alone is measured over a
    wide range of arguments."""
    announce(f"epilogue exact products M={M} {act}")
    K, N = 256, 272
    rng = np.random.default_rng(M)
    codes = rng.integers(1, 16, (K, N)).astype(np.uint8)
    one = np.full((K // 128, N), 0x3F80, np.uint16)
    packed, scales = q4.pack_native(codes, one)
    a = np.zeros((M, K), np.float32)
    a[np.arange(M), rng.integers(0, K, M)] = rng.choice([0.0078125, 0.125, 0.5, 1.0, 3.0, 20.0], M)
    bias = synth.normal_bf16((N,), 2)
    res = f32_to_bf16_bits(bf16_bits_to_f32(synth.normal_bf16((M, N), 3)) * np.float32(2.0 ** -10))
    product = a.astype(np.float64) @ (codes.astype(np.float64) - 8)
    d_p = torch.from_numpy(packed.view(np.int32)).cuda()
    d_s = torch.from_numpy(scales.view(np.int16)).cuda()
    lin = ops.W4A16Linear(ops.Int4G128Weight(d_p, d_s, K, N), dev_bf16(bias), act)
    for with_res in (False, True):
        y = lin(dev_bf16(f32_to_bf16_bits(a)), residual=dev_bf16(res) if with_res else None)
        torch.cuda.synchronize()
        x = product + f64(bias)
        inner = block.activation(x, act)
        ref = inner + (f64(res) if with_res else 0.0)
        size = np.abs(inner) + (np.abs(f64(res)) if with_res else 0.0)
        tiny = 2.0 ** -24 * np.abs(x) * (np.abs(inner) > 0) * EPI + 2.0 ** -120
        err = np.abs(f64(host_bits16(y)) - ref)
        assert (err <= 2.0 ** -8 * np.abs(ref) * (1 + 2.0 ** -8) + EPI * size + tiny).all(), float((err / size).max())


def test_refusals(ops):
    announce("epilogue refusals")
    wt, _ = weight(ops, 512, 512)
    a = dev_bf16(synth.activations(4, 512, seed=1))
    with pytest.raises(ValueError):
        ops.W4A16Linear(wt, activation="tanh")
    with pytest.raises(ValueError):
        ops.W4A16Linear(wt, bias=torch.zeros(8, dtype=torch.bfloat16, device="cuda:0"))
    with pytest.raises(TypeError):
        ops.W4A16Linear(wt, bias=torch.zeros(512, device="cuda:0"))
    with pytest.raises(ValueError):
        ops.W4A16Linear(wt)(a, residual=torch.zeros((3, 512), dtype=torch.bfloat16, device="cuda:0"))
    with pytest.raises(ops.QGemmError):
        ops.qgemm_w4a16_epilogue(a, wt.packed, wt.scales, None, 5, None, torch.empty_like(a), 4, 512, 512)


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_bias_at_any_word(ops, M, N, K):
    """A bias that starts at any 4-byte word gives the bits of an aligned one; at a
    half word it is refused."""
    announce(f"bias alignment M={M} N={N} K={K}")
    wt, _ = weight(ops, K, N)
    a = dev_bf16(synth.activations(M, K, seed=1))
    room = torch.zeros(N + 16, dtype=torch.bfloat16, device="cuda:0")
    bias = dev_bf16(synth.normal_bf16((N,), 2))
    want = ops.W4A16Linear(wt, bias, "silu")(a)
    for off in (2, 6):
        part = room[off:off + N]
        part.copy_(bias)
        got = ops.W4A16Linear(wt, part, "silu")(a)
        torch.cuda.synchronize()
        assert torch.equal(got, want), off
    with pytest.raises(ops.QGemmError):
        ops.W4A16Linear(wt, room[1:1 + N], "silu")(a)


@pytest.mark.parametrize("M,N,K", [s for s in SHAPES if s in ((16, 1024, 14336), (12, 272, 16384), (100, 4096, 4096),
                                                              (130, 8192, 8192))])
def test_split_slots_are_written_before_they_are_read(ops, M, N, K):
    """K splits: the partial sums' memory holds NaN before every call, the inputs
    alternate, and one workspace serves the plain product and the epilogue in turn."""
    announce(f"epilogue on a spoilt workspace M={M} N={N} K={K}")
    assert not ops.w4a16_kernel_for(M, N, K).endswith("S=1")
    wt, _ = weight(ops, K, N)
    bias, res = dev_bf16(synth.normal_bf16((N,), 2)), dev_bf16(synth.normal_bf16((M, N), 3))
    ins = [dev_bf16(synth.activations(M, K, seed=s)) for s in (1, 2)]
    lin = ops.W4A16Linear(wt)
    ws, need = lin.workspace(M)
    want = {}
    for turn in range(6):
        i = turn % 2
        ws[64 * 1024:].fill_(0xFF)
        y = torch.empty((M, N), dtype=torch.bfloat16, device="cuda:0")
        ops.qgemm_w4a16_epilogue(ins[i], wt.packed, wt.scales, bias, "gelu", res, y, M, N, K, ws, need)
        p = lin(ins[i])
        torch.cuda.synchronize()
        assert bool(torch.isfinite(y).all()) and not bool(ws[:64 * 1024].any())
        if i in want:
            assert torch.equal(y, want[i][0]) and torch.equal(p, want[i][1])
        want[i] = (y, p)


def test_no_rows(ops):
    announce("epilogue M=0")
    wt, _ = weight(ops, 512, 512)
    empty = torch.empty((0, 512), dtype=torch.bfloat16, device="cuda:0")
    assert ops.W4A16Linear(wt, activation="relu")(empty, residual=empty).shape == (0, 512)
