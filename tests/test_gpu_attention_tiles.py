"""paged_attention of many rows: every number of key tiles from one on, positions without pages inside the sequences, and
values that are not finite in several tiles while the scores grow from tile to tile."""
import numpy as np
import pytest
import torch

from attention_helpers import Batch, attend, bf16, check
from gpu_helpers import announce
from oracle import attention as oracle

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ops():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    from weight_only_quantized_w4a16_amd import ops as _ops
    return _ops


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("D", [64, 128])
def test_every_number_of_tiles(ops, D, fmt):
    for kv in (70, 128, 129, 192, 256, 257, 330, 400, 511, 600):
        b = Batch([70], [kv], 2, 1, D, 16, fmt, seed=kv)
        want = oracle.paged_attention(b.q, b.k, b.v, b.table, b.q_offsets, b.kv_len, D ** -0.5)
        announce(f"tiles of {kv} keys {fmt} D={D}")
        out, lse = attend(ops, b, max_q=70)
        check(b, out, lse, want, f"{kv} keys")


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("window,sinks", [(0, 0), (300, 70)])
def test_many_tiles_without_a_split(ops, D, fmt, window, sinks):
    """Row tiles enough to fill the GPU, so that a workgroup goes over all keys of its rows: up to 18 tiles."""
    b = Batch([900], [1150], 64, 64, D, 64, fmt, seed=D)
    some = slice(3, None, 30)
    want = oracle.paged_attention(b.q[:, some], b.k[:, some], b.v[:, some], b.table, b.q_offsets, b.kv_len, D ** -0.5, window, sinks)
    announce(f"many tiles {fmt} D={D} window={window}")
    out, lse = attend(ops, b, window=window, sinks=sinks, max_q=900)
    check(b, out[:, some], lse[:, some], want, f"window={window}")


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("page", [16, 64])
@pytest.mark.parametrize("window,sinks", [(0, 0), (150, 20)])
def test_positions_without_pages(ops, D, fmt, page, window, sinks):
    """Entries below zero and past the last page hold no keys: in the middle, at the ends, and a whole sequence of them."""
    b = Batch([90, 66, 80], [500, 300, 100], 4, 2, D, page, fmt, seed=D + page)
    b.table[0, 0], b.table[0, 2], b.table[0, 250 // page], b.table[0, 499 // page] = -1, b.pages, -7, 2 ** 31 - 1
    b.table[1, 64 // page:192 // page] = -1
    b.table[2, :] = b.pages
    want = oracle.paged_attention(b.q, b.k, b.v, b.table, b.q_offsets, b.kv_len, D ** -0.5, window, sinks)
    assert (want[1][-80:] == -np.inf).all()
    for m in (0, 90):
        announce(f"missing pages {fmt} D={D} page={page} window={window} max_q={m}")
        out, lse = attend(ops, b, window=window, sinks=sinks, max_q=m)
        check(b, out, lse, want, f"max_q={m}")


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("D", [64, 128])
def test_values_that_are_not_finite_under_growing_scores(ops, D, fmt):
    """Under a window of 70 every row's first and last tile hold values that it does not see, some of them not finite, and
    the keys grow with the position, so sums of such tiles are rescaled."""
    b = Batch([200], [500], 2, 1, D, 16, fmt, seed=11)
    along = 0.2 + np.arange(500) / 100
    for p in range(500):
        page, slot = b.table[0, p // 16], p % 16
        b.k[page, :, slot] *= along[p]
        if fmt == "e4m3":
            b.k_scale_t[page, :, slot] *= float(along[p])
    if fmt == "bf16":
        b.k, b.k_t = bf16(b.k)
    else:                                                # the scales were rounded
        from oracle import fp8_e4m3 as f8
        with np.errstate(invalid="ignore"):
            b.k = f8.e4m3_decode(b.k_t.numpy()).astype(np.float64) * b.k_scale_t.double().numpy()[..., None]
    for i, p in enumerate(range(235, 500, 37)):
        page, slot, e = b.table[0, p // 16], p % 16, (5 * i) % D
        if fmt == "bf16":
            b.v[page, :, slot, e] = b.v_t[page, :, slot, e] = [float("nan"), float("inf")][i % 2]
        else:
            b.v[page, :, slot, e], b.v_t[page, :, slot, e] = np.nan, 0x7f
    want = oracle.paged_attention(b.q, b.k, b.v, b.table, b.q_offsets, b.kv_len, D ** -0.5, 70, 0)
    y, l64, mean, reach = want
    fine = np.isfinite(y)
    assert fine.any(0).all() and not fine.all(1).all()
    announce(f"odd values, growing scores {fmt} D={D}")
    out, lse = attend(ops, b, window=70, max_q=200)
    got = out.double().cpu().numpy()
    assert np.array_equal(np.isfinite(got), fine), np.argwhere(np.isfinite(got) != fine)[:5]
    # as in check(), where the values are finite
    x = (2 * (D + 4) + 8) * 2.0 ** -24 * reach
    rel = np.expm1(2 * x) + 2.0 ** -8 + 2.0 ** -20 + 500 * 2.0 ** -23
    bound = rel[..., None] * np.where(fine, mean, 0) + 2.0 ** -8 * (1 + 2.0 ** -6) * np.abs(np.where(fine, y, 0)) + 1e-30
    with np.errstate(invalid="ignore"):
        err = np.where(fine, np.abs(got - y), 0)
    assert (err <= bound).all(), float((err / bound).max())
    lb = 2 * x + 2.0 ** -20 + 500 * 2.0 ** -23 + 2.0 ** -22 * np.abs(l64)
    assert (np.abs(lse.double().cpu().numpy() - l64) <= lb).all()
