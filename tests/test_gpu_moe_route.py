"""moe_dispatch, moe_gather, moe_combine and their gradient against the oracle.

The sort and the copies are exact.  combine: fp32 fused multiply-adds in slot
order and one rounding to bf16; drows: one fp32 product, one rounding; dweights:
an fp32 sum.  The bounds are in each test.
"""
import numpy as np
import pytest
import torch

from gpu_helpers import announce, dev_bf16, host_bits16
from oracle import block
from oracle.bf16 import bf16_bits_to_f32, f32_to_bf16_bits
from weight_only_quantized_w4a16_amd import synth

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ops():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    from weight_only_quantized_w4a16_amd import ops as _ops
    return _ops


def f64(bits):
    return bf16_bits_to_f32(bits).astype(np.float64)


def route(ids, E):
    """oracle.block.route by one stable argsort (the same result; large batches)."""
    flat = ids.reshape(-1).astype(np.int64)
    kept = (flat >= 0) & (flat < E)
    key = np.where(kept, flat, E)
    order = np.argsort(key, kind="stable")
    row = np.empty(flat.size, np.int32)
    row[order] = np.arange(flat.size, dtype=np.int32)
    row[~kept] = -1
    offsets = np.searchsorted(key[order], np.arange(E + 1)).astype(np.int32)
    return offsets, row.reshape(ids.shape)


def make_ids(B, k, E, kind, seed):
    rng = np.random.default_rng(seed)
    if kind == "uniform":
        return rng.integers(0, E, (B, k)).astype(np.int32)         # a token may name an expert twice
    if kind == "one expert":
        return np.full((B, k), E - 1, np.int32)
    if kind == "none":
        return np.full((B, k), -1, np.int32)
    ids = rng.integers(0, E, (B, k)).astype(np.int32)              # "dropped": ids outside [0, E) of every kind
    bad = np.array([-1, E, E + 5, -(2 ** 31), 2 ** 31 - 1], np.int64).astype(np.int32)
    drop = rng.random((B, k)) < 0.3
    ids[drop] = rng.choice(bad, drop.sum())
    return ids


def dispatch(ops, ids, E, rows=None, scale=None):
    """Raw call into buffers of a known content; returns offsets, row_of_slot, rows, scales (host)."""
    B, k = ids.shape
    T = B * k
    di = torch.from_numpy(ids).cuda()
    offsets = torch.full((E + 1 + 8,), 77, dtype=torch.int32, device="cuda:0")
    row = torch.full((T + 8,), 77, dtype=torch.int32, device="cuda:0")
    need = ops.moe_dispatch_workspace_bytes(B, k, E)
    ws = torch.full((need + 64,), 0x7F, dtype=torch.uint8, device="cuda:0")
    out = so = None
    width = 0
    if rows is not None:
        width = rows.shape[1] * rows.element_size()
        out = torch.full((T + 1, width), 0x5A, dtype=torch.uint8, device="cuda:0")
    if scale is not None:
        so = torch.full((T + 1,), -7.0, dtype=torch.float32, device="cuda:0")
    ops.moe_dispatch(di, rows, scale, B, k, E, width, offsets, row, out, so, ws, need)
    torch.cuda.synchronize()
    assert bool((ws[need:] == 0x7F).all()) and bool((offsets[E + 1:] == 77).all()) and bool((row[T:] == 77).all())
    if out is not None:
        assert bool((out[T] == 0x5A).all())
    if so is not None:
        assert float(so[T]) == -7.0
    return (offsets[:E + 1].cpu().numpy(), row[:T].cpu().numpy().reshape(B, k),
            None if out is None else out[:T].cpu().numpy(), None if so is None else so[:T].cpu().numpy())


SORTS = [(1, 1, 1), (1, 8, 128), (2, 3, 5), (4, 8, 128), (16, 8, 128), (31, 2, 1024), (64, 4, 60), (100, 5, 3),
         (128, 8, 128), (257, 8, 128), (511, 4, 64), (1000, 3, 1024), (4099, 8, 256), (9000, 1, 7), (70001, 4, 65),
         (300, 17, 40), (700, 9, 128), (1048577, 1, 64), (300000, 4, 1024)]


@pytest.mark.parametrize("B,k,E", SORTS)
@pytest.mark.parametrize("kind", ["uniform", "one expert", "none", "dropped"])
def test_sort(ops, B, k, E, kind):
    announce(f"moe_dispatch sort B={B} k={k} E={E} {kind}")
    ids = make_ids(B, k, E, kind, B + k + E)
    offsets, row, _, _ = dispatch(ops, ids, E)
    want_off, want_row = route(ids, E)
    if B * k <= 600:
        for a, b in zip((want_off, want_row), block.route(ids, E)):
            assert np.array_equal(a, b)
    assert np.array_equal(offsets, want_off)
    assert np.array_equal(row, want_row)


# row bytes: one piece of 8 or 16 bytes up to several workgroups a row, 8-byte pieces where 16 does not divide
WIDTHS = [8, 16, 24, 768, 1032, 2048, 4096, 4104, 8192, 28672]


@pytest.mark.parametrize("width", WIDTHS)
@pytest.mark.parametrize("B,k,E,kind", [(1, 8, 128, "uniform"), (5, 3, 4, "dropped"), (33, 8, 16, "dropped"),
                                        (700, 2, 60, "uniform"), (500, 8, 128, "dropped"), (600, 8, 128, "uniform")])
def test_dispatch_rows(ops, width, B, k, E, kind):
    announce(f"moe_dispatch rows width={width} B={B} k={k} E={E} {kind}")
    rng = np.random.default_rng(width + B)
    ids = make_ids(B, k, E, kind, width)
    x = rng.integers(0, 256, (B, width)).astype(np.uint8)
    s = rng.standard_normal(B).astype(np.float32)
    dx, ds = torch.from_numpy(x).cuda(), torch.from_numpy(s).cuda()
    offsets, row, out, so = dispatch(ops, ids, E, dx, ds)
    want_off, want_row = route(ids, E)
    assert np.array_equal(offsets, want_off) and np.array_equal(row, want_row)
    blank = np.full((B * k, width), 0x5A, np.uint8)
    assert np.array_equal(out, block.gather(x, want_row, blank))   # rows of no slot keep their contents
    assert np.array_equal(so, block.gather(s, want_row, np.full(B * k, -7.0, np.float32)))
    # the same copies by the row numbers alone
    rows2 = torch.full((B * k, width), 0x5A, dtype=torch.uint8, device="cuda:0")
    s2 = torch.full((B * k,), -7.0, device="cuda:0")
    ops.moe_gather(dx, ds, torch.from_numpy(row).cuda(), B, k, width, rows2, s2)
    torch.cuda.synchronize()
    assert np.array_equal(rows2.cpu().numpy(), out) and np.array_equal(s2.cpu().numpy(), so)


def test_dispatch_no_tokens(ops):
    announce("moe_dispatch B=0")
    offsets, row, _, _ = dispatch(ops, np.empty((0, 8), np.int32), 1024)
    assert not offsets.any() and row.size == 0


COMBINES = [(1, 8, 128, 2048), (1, 1, 1, 8), (5, 3, 4, 24), (16, 8, 128, 2048), (33, 8, 16, 2056), (40, 11, 7, 512),
            (3, 2, 8, 28672), (130, 4, 60, 1000), (65, 17, 5, 64)]


def routed(B, k, E, K, kind, seed):
    ids = make_ids(B, k, E, kind, seed)
    row = route(ids, E)[1]
    rng = np.random.default_rng(seed)
    rows = synth.normal_bf16((B * k, K), seed)
    spare = np.setdiff1d(np.arange(B * k), row[row >= 0])
    rows[spare] = 0x7FC0                                            # rows of no slot: NaN, never to be read
    w = rng.random((B, k)).astype(np.float32)
    w[row < 0] = np.nan                                             # nor the weights of slots without a row
    return row, rows, w


@pytest.mark.parametrize("B,k,E,K", COMBINES)
@pytest.mark.parametrize("weighted", [True, False])
@pytest.mark.parametrize("residual", [True, False])
def test_combine(ops, B, k, E, K, weighted, residual):
    """|y - y64| <= half a bf16 step + (k + 1) fp32 roundings of the sum of the terms' absolute values."""
    announce(f"moe_combine B={B} k={k} E={E} K={K} weighted={weighted} residual={residual}")
    row, rows, w = routed(B, k, E, K, "dropped", B + K)
    res = synth.normal_bf16((B, K), 9) if residual else None
    y = torch.full((B + 1, K), 7.0, dtype=torch.bfloat16, device="cuda:0")
    d_row = torch.from_numpy(row).cuda()
    d_w = torch.from_numpy(w).cuda() if weighted else None
    d_res = dev_bf16(res) if residual else None
    ops.moe_combine(dev_bf16(rows), d_row, d_w, d_res, B, k, K, y)
    torch.cuda.synchronize()
    assert bool((y[B] == 7.0).all())
    w64 = w.astype(np.float64) if weighted else None
    r64 = f64(res) if residual else None
    ref = block.combine(f64(rows), row, w64, r64)
    size = block.combine(np.abs(f64(rows)), row, w64, np.abs(r64) if residual else None)
    got = f64(host_bits16(y[:B]))
    assert (np.abs(got - ref) <= 2.0 ** -8 * np.abs(ref) * (1 + 2.0 ** -8) + (k + 1) * 2.0 ** -24 * size * 2).all()
    if residual:                                                    # the residual's own memory: the same bits
        ops.moe_combine(dev_bf16(rows), d_row, d_w, d_res, B, k, K, d_res)
        torch.cuda.synchronize()
        assert torch.equal(d_res, y[:B])


@pytest.mark.parametrize("B,k,E,K", COMBINES)
@pytest.mark.parametrize("weighted", [True, False])
def test_combine_backward(ops, B, k, E, K, weighted):
    """drows exactly the rounding of the fp32 product.  dweights: an fp32 sum of K
    terms, each thread's share at most 8 ceil(K / 2048) terms long, then 6 + 4
    partial sums: |error| <= (8 ceil(K / 2048) + 11) 2^-24 sum |dy row|."""
    announce(f"moe_combine_backward B={B} k={k} E={E} K={K} weighted={weighted}")
    row, rows, w = routed(B, k, E, K, "dropped", B + K + 1)
    dy = synth.normal_bf16((B, K), 4)
    d_dy, d_rows, d_row = dev_bf16(dy), dev_bf16(rows), torch.from_numpy(row).cuda()
    d_w = torch.from_numpy(w).cuda() if weighted else None
    drows = torch.full((B * k + 1, K), 7.0, dtype=torch.bfloat16, device="cuda:0")
    dw = torch.full((B * k + 1,), 7.0, device="cuda:0")
    ops.moe_combine_backward(d_dy, d_rows, d_row, d_w, B, k, K, drows, dw)
    torch.cuda.synchronize()
    assert bool((drows[B * k] == 7.0).all()) and float(dw[B * k]) == 7.0
    want = np.full((B * k, K), 7.0, np.float32)
    for b, j in zip(*np.nonzero(row >= 0)):
        want[row[b, j]] = bf16_bits_to_f32(dy[b]) * (w[b, j] if weighted else np.float32(1))
    assert np.array_equal(host_bits16(drows[:B * k]), f32_to_bf16_bits(want))
    _, dw64 = block.combine_backward(f64(dy), f64(rows), row, w.astype(np.float64))
    size = block.combine_backward(np.abs(f64(dy)), np.abs(f64(rows)), row, None)[1]
    got = dw[:B * k].cpu().numpy().reshape(B, k).astype(np.float64)
    bound = (8 * -(-K // 2048) + 11) * 2.0 ** -24 * size
    assert (np.abs(got - dw64) <= bound + 2.0 ** -149).all()
    assert not got[row < 0].any()
    # either output alone: the same
    drows2, dw2 = torch.full_like(drows, 7.0), torch.full_like(dw, 7.0)
    ops.moe_combine_backward(d_dy, None, d_row, d_w, B, k, K, drows2, None)
    ops.moe_combine_backward(d_dy, d_rows, d_row, d_w, B, k, K, None, dw2)
    torch.cuda.synchronize()
    assert torch.equal(drows2, drows) and torch.equal(dw2, dw)


def test_gradient_against_differences(ops):
    """The kernels' gradients against central differences of the oracle's combine
    (linear in rows and in weights: the differences are exact up to fp64)."""
    announce("moe gradient against differences")
    B, k, E, K = 6, 3, 4, 32
    row, rows, w = routed(B, k, E, K, "dropped", 3)
    rows = np.where((np.arange(B * k)[:, None] < (row >= 0).sum()), rows, np.uint16(0))
    w = np.where(row >= 0, w, 0).astype(np.float32)
    dy = synth.normal_bf16((B, K), 5)
    r = ops.MoeRouting(None, torch.from_numpy(row).cuda())
    drows, dw = r.combine_backward(dev_bf16(dy), dev_bf16(rows), torch.from_numpy(w).cuda())
    dx = r.combine(dev_bf16(rows))                                   # gradient of the gather, for drows = rows
    torch.cuda.synchronize()
    loss = lambda rr, ww: float((block.combine(rr, row, ww, None) * f64(dy)).sum())
    R, W = f64(rows), w.astype(np.float64)
    rng = np.random.default_rng(0)
    for _ in range(20):
        b, j = rng.integers(B), rng.integers(k)
        e = np.zeros_like(W)
        e[b, j] = 0.5
        num = loss(R, W + e) - loss(R, W - e)
        assert abs(num - float(dw[b, j])) <= 1e-5 * (1 + abs(num))
        if row[b, j] < 0:
            continue
        c = rng.integers(K)
        e = np.zeros_like(R)
        e[row[b, j], c] = 0.5
        num = loss(R + e, W) - loss(R - e, W)
        assert abs(num - float(drows[row[b, j], c])) <= 2.0 ** -8 * abs(num) * (1 + 2.0 ** -8)
        # d/dx[b, c] of <gather(x), rows>
        x = np.zeros((B, K))
        x[b, c] = 0.5
        g = block.gather(x, row, np.zeros((B * k, K)))
        num = 2 * float((g * R)[: (row >= 0).sum()].sum())
        assert abs(num - float(dx[b, c])) <= 2.0 ** -8 * abs(num) + k * 2.0 ** -23 * 8


def test_malformed_row_numbers_stay_in_bounds(ops):
    """Entries outside 0 .. B k - 1 are no rows."""
    announce("moe malformed row numbers")
    B, k, K = 8, 4, 64
    row = np.arange(B * k, dtype=np.int32).reshape(B, k)
    row[::2, 1] = np.array([B * k, -2, 2 ** 31 - 1, -(2 ** 31)], np.int32)
    rows, x = synth.normal_bf16((B * k, K), 1), synth.normal_bf16((B, K), 2)
    d_row = torch.from_numpy(row).cuda()
    ok = np.where((row >= 0) & (row < B * k), row, -1)
    y = torch.empty((B, K), dtype=torch.bfloat16, device="cuda:0")
    ops.moe_combine(dev_bf16(rows), d_row, None, None, B, k, K, y)
    out = torch.zeros((B * k, K), dtype=torch.bfloat16, device="cuda:0")
    ops.moe_gather(dev_bf16(x), None, d_row, B, k, 2 * K, out, None)
    dw = torch.empty((B, k), device="cuda:0")
    ops.moe_combine_backward(dev_bf16(x), dev_bf16(rows), d_row, None, B, k, K, None, dw)
    torch.cuda.synchronize()
    assert not np.isnan(f64(host_bits16(y))).any()
    assert np.array_equal(host_bits16(out), block.gather(x, ok, np.zeros((B * k, K), np.uint16)))
    assert not dw.cpu().numpy()[ok < 0].any() and dw.cpu().numpy()[ok >= 0].all()


def test_helpers_refusals(ops):
    announce("moe helpers: refusals")
    ids = torch.zeros((4, 2), dtype=torch.int32, device="cuda:0")
    x = torch.zeros((4, 64), dtype=torch.bfloat16, device="cuda:0")
    with pytest.raises(TypeError):
        ops.MoeRouting.dispatch(ids.long(), 8, x)
    with pytest.raises(ValueError):
        ops.MoeRouting.dispatch(ids, 8, x[:3])
    with pytest.raises(ValueError):
        ops.MoeRouting.dispatch(ids, 8, None, torch.ones(4, device="cuda:0"))
    with pytest.raises(ops.QGemmError):
        ops.MoeRouting.dispatch(ids, 1025, x)
    r, rows, s = ops.MoeRouting.dispatch(ids, 8, x)
    assert s is None and rows.shape == (8, 64)
    with pytest.raises(ValueError):
        r.combine(rows[:7])
    with pytest.raises(TypeError):
        r.combine(rows, weights=torch.ones((4, 2), dtype=torch.bfloat16, device="cuda:0"))
    with pytest.raises(ValueError):
        r.combine(rows, residual=x[:, :32].contiguous())
    with pytest.raises(ValueError):
        r.combine_backward(x[:2], rows)
    torch.cuda.synchronize()


def test_rows_past_32_bit_offsets(ops):
    """Routed rows of more than 2^31 elements: the last rows and their way back."""
    B, k, E, K = 34_000, 8, 8, 8192
    announce(f"moe rows past 32-bit offsets B={B} k={k} K={K}")
    ids = np.tile(np.arange(k, dtype=np.int32), (B, 1))
    x = torch.zeros((B, K), dtype=torch.bfloat16, device="cuda:0")
    tail = synth.normal_bf16((2, K), 1)
    x[-2:] = dev_bf16(tail)
    r, rows, _ = ops.MoeRouting.dispatch(torch.from_numpy(ids).cuda(), E, x)
    y = r.combine(rows, residual=x)
    torch.cuda.synchronize()
    assert torch.equal(rows[B * k - 2:], x[-2:]) and torch.equal(rows[B - 2:B], x[-2:])
    assert not bool(y[:-2].any())
    assert np.array_equal(host_bits16(y[-2:]), f32_to_bf16_bits(bf16_bits_to_f32(tail) * 9))
    drows, dw = r.combine_backward(x, rows)
    torch.cuda.synchronize()
    assert torch.equal(drows[B * k - 2:], x[-2:]) and not bool(dw[:-2].any()) and bool((dw[-2:] > 0).all())
