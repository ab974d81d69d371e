"""paged_attention against the oracle in 64 bits: head layouts, cache types, page sizes, ragged batches, windows with first
positions that stay visible, positions without pages, and rows that see nothing."""
import numpy as np
import pytest
import torch

from attention_helpers import Batch, attend, check
from gpu_helpers import announce
from oracle import attention as oracle

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ops():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    from weight_only_quantized_w4a16_amd import ops as _ops
    return _ops


def verify(ops, b, what, scale=None, window=0, sinks=0, shared=0):
    """Every kernel that the call may choose: by an unknown max_q, the real one, and one that is too small."""
    want = oracle.paged_attention(b.q, b.k, b.v, b.table, b.q_offsets, b.kv_len, scale or b.D ** -0.5, window, sinks)
    for m in (0, int(np.diff(b.q_offsets).max()), 1):
        announce(f"{what} max_q={m}")
        out, lse = attend(ops, b, scale, window, sinks, shared, m)
        check(b, out, lse, want, f"{what} max_q={m}")


# (new tokens, positions) of each sequence
BATCHES = {
    "one key": ([1], [1]),
    "decode": ([1, 1, 1, 1], [1, 17, 128, 301]),
    "with padding": ([1, 0, 1, 2], [33, 0, 0, 2]),                # no tokens; no positions; and all of them new
    "few tokens each": ([3, 1, 7, 2], [3, 129, 40, 64]),
    "more tokens than positions": ([6, 4], [3, 0]),
    "prefill": ([70], [200]),
}


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("batch", BATCHES)
def test_batches(ops, batch, D, fmt):
    new, kv = BATCHES[batch]
    for (Hq, Hkv), page in (((4, 2), 16), ((10, 2), 64), ((3, 3), 256)):
        b = Batch(new, kv, Hq, Hkv, D, page, fmt, seed=D + Hq, extra_tokens=2)
        verify(ops, b, f"{batch} {fmt} D={D} Hq={Hq} Hkv={Hkv} page={page}")


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 3), (16, 0), (31, 1), (64, 4), (129, 200), (1 << 30, 5)])
def test_windows(ops, window, sinks, fmt):
    b = Batch([1, 1, 4, 40, 1], [700, 90, 333, 260, 5], 8, 2, 64, 16, fmt, seed=window)
    verify(ops, b, f"window {window} sinks {sinks} {fmt}", window=window, sinks=sinks)


@pytest.mark.parametrize("Hq,Hkv", [(32, 8), (32, 4), (64, 8), (16, 16), (8, 1), (7, 1), (40, 2)])
def test_head_layouts(ops, Hq, Hkv):
    b = Batch([1, 2, 1], [1030, 77, 600], Hq, Hkv, 128, 32, seed=Hq)
    verify(ops, b, f"Hq={Hq} Hkv={Hkv}")


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_many_sequences(ops, fmt):
    rng = np.random.default_rng(5)
    kv = rng.integers(0, 60, 150)
    new = [int(rng.integers(0, 3)) for _ in kv]
    b = Batch(new, kv.tolist(), 2, 1, 64, 16, fmt, seed=9)
    verify(ops, b, f"150 sequences {fmt}")


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("new,kv", [([130], [130]), ([65, 3, 200], [400, 300, 200]), ([33, 1, 0, 17], [33, 500, 70, 1100])])
def test_prefill(ops, new, kv, D, fmt):
    for Hq, Hkv, page in ((6, 2, 16), (8, 1, 64), (2, 2, 128)):
        b = Batch(new, kv, Hq, Hkv, D, page, fmt, seed=D + Hq, extra_tokens=3)
        verify(ops, b, f"prefill {new} {kv} {fmt} D={D} Hq={Hq} Hkv={Hkv} page={page}")
        verify(ops, b, f"prefill {new} {kv} {fmt} D={D} Hq={Hq} Hkv={Hkv} page={page} windowed", window=50, sinks=3)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("prefix,page", [(16, 16), (48, 16), (256, 256), (640, 64)])
def test_shared_prefix(ops, prefix, page, fmt):
    """The same as without it, also where a sequence's new tokens lie inside the prefix or where it has none."""
    for new, more, D in (([1] * 5, [1, 9, 40, 2, 300], 128), ([2, 4, 1], [2, 70, 33], 64), ([40, 1, 0, 5], [50, 1, 0, 5], 64)):
        kv = [prefix + m for m in more]
        b = Batch(new, kv, 8, 2, D, page, fmt, seed=prefix + len(new), extra_tokens=1, shared=prefix)
        want_table = b.table.copy()
        b.table[1:, :prefix // page] = -1                # not read
        want = oracle.paged_attention(b.q, b.k, b.v, want_table, b.q_offsets, b.kv_len, D ** -0.5)
        for m in (0, max(new)):
            what = f"shared {prefix} page {page} {fmt} new={new} max_q={m}"
            announce(what)
            out, lse = attend(ops, b, shared=prefix, max_q=m)
            check(b, out, lse, want, what)
        windowed = oracle.paged_attention(b.q, b.k, b.v, want_table, b.q_offsets, b.kv_len, D ** -0.5, 60, 5)
        out, lse = attend(ops, b, shared=prefix, window=60, sinks=5)
        check(b, out, lse, windowed, "windowed")
    short = Batch([3, 1, 2], [prefix, 0, prefix + 20], 4, 2, 64, page, fmt, seed=1, shared=prefix)
    want = oracle.paged_attention(short.q, short.k, short.v, short.table, short.q_offsets, short.kv_len, 0.125)
    out, lse = attend(ops, short, shared=prefix)
    check(short, out, lse, want, "new tokens inside the prefix")


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("D,Hkv,prefix,page", [(128, 8, 2048, 64), (64, 4, 8192, 256), (128, 8, 2064, 16)])
def test_shared_prefix_in_a_pass_of_its_own(ops, D, Hkv, prefix, page, fmt):
    """Prefixes whose rereading a pass of its own spares (from 64 MB of bf16 on): parts of the prefix joined with a
    sequence's own, in both kernels; windows; new tokens inside the prefix; sequences without positions."""
    assert 8 * prefix * Hkv * D * 4 >= 64 << 20
    for new, more in (([1] * 9, [1, 300, 2, 17, 64, 129, 5, 1, 40]), ([12, 1, 30, 0, 2, 1, 1, 1, 17], [12, 1, 700, 5, 2, 90, 33, 1, 17])):
        kv = [prefix + m for m in more]
        b = Batch(new, kv, Hkv, Hkv, D, page, fmt, seed=prefix + len(new), extra_tokens=1, shared=prefix)
        want_table = b.table.copy()
        b.table[1:, :prefix // page] = -1                    # not read
        need = ops.paged_attention_workspace_bytes(b.T, b.B, b.width, Hkv, Hkv, D, page, prefix, 0)
        assert need > 65536 + b.T * Hkv * D * 4              # parts of the prefix
        want = oracle.paged_attention(b.q, b.k, b.v, want_table, b.q_offsets, b.kv_len, D ** -0.5)
        for m in (0, max(new)):
            announce(f"shared {prefix} {fmt} new={new} max_q={m}")
            out, lse = attend(ops, b, shared=prefix, max_q=m)
            check(b, out, lse, want, f"shared {prefix} {fmt} max_q={m}")
    want = oracle.paged_attention(b.q, b.k, b.v, want_table, b.q_offsets, b.kv_len, D ** -0.5, 100, 70)
    out, lse = attend(ops, b, shared=prefix, window=100, sinks=70)
    check(b, out, lse, want, "windowed")
    short = Batch([3, 1, 2, 1, 1, 1, 1, 1, 90], [prefix, 0, prefix + 20, 3, prefix - 5, 1, 2, prefix, prefix + 10], Hkv, Hkv, D, page, fmt,
                  seed=1, shared=prefix)
    want = oracle.paged_attention(short.q, short.k, short.v, short.table, short.q_offsets, short.kv_len, D ** -0.5)
    for m in (0, 90):
        out, lse = attend(ops, short, shared=prefix, max_q=m)
        check(short, out, lse, want, "new tokens inside the prefix")


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("new,kv,window", [([5], [20], 0), ([90, 3], [150, 130], 0), ([90], [150], 16), ([4, 1], [200, 9], 16)])
def test_values_that_are_not_finite_reach_only_rows_that_see_them(ops, fmt, new, kv, window):
    """Infinite and NaN values (and, in 8 bits, a NaN code and an infinite scale) at a few positions: rows that see one are
    not finite in its elements, all others are as if they were not there."""
    b = Batch(new, kv, 4, 2, 64, 16, fmt, seed=7)
    spots = []                                               # (sequence, position, element)
    for s, n in enumerate(kv):
        for p in {n - 1, n - 2, max(0, n - new[s] // 2), max(0, n - 40)}:
            spots.append((s, p, int((7 * p + 3) % 64)))
    for i, (s, p, e) in enumerate(spots):
        page, slot = b.table[s, p // 16], p % 16
        if fmt == "bf16":
            x = [float("inf"), float("-inf"), float("nan")][i % 3]
            b.v[page, :, slot, e] = x
            b.v_t[page, :, slot, e] = x
        elif p < kv[s] - 1:
            b.v[page, :, slot, e] = np.nan
            b.v_t[page, :, slot, e] = 0x7f
        else:
            b.v_scale_t[page, :, slot] = float("inf")        # the whole row: infinities, NaN where the code is zero
            b.v[page, :, slot] = np.inf
    want, l64, mean, reach = oracle.paged_attention(b.q, b.k, b.v, b.table, b.q_offsets, b.kv_len, 0.125, window, 0)
    fine = np.isfinite(want)
    assert fine.any() and not fine.all()
    for m in (0, max(new)):
        announce(f"values {fmt} {new} {kv} window {window} max_q={m}")
        out, lse = attend(ops, b, 0.125, window=window, max_q=m)
        got = out.double().cpu().numpy()
        assert np.array_equal(np.isfinite(got), fine), np.argwhere(np.isfinite(got) != fine)[:5]
        lim = 2.0 ** -7 * np.where(fine, mean, 0) + 2.0 ** -8 * np.abs(np.where(fine, want, 0)) + 1e-6
        with np.errstate(invalid="ignore"):
            assert (np.abs(np.where(fine, got - want, 0)) <= lim).all()


def test_keys_that_are_not_finite(ops):
    """A NaN key makes the rows that see it NaN, an infinite one those whose scores it leaves infinite; the others stay."""
    for new, kv in (([3], [40]), ([80], [140])):
        b = Batch(new, kv, 2, 1, 64, 16, seed=2)
        p = kv[0] - 2
        page, slot = b.table[0, p // 16], p % 16
        b.k[page, :, slot, 5] = np.nan
        b.k_t[page, :, slot, 5] = float("nan")
        want = oracle.paged_attention(b.q, b.k, b.v, b.table, b.q_offsets, b.kv_len, 0.125)
        out, lse = attend(ops, b, 0.125)
        got = out.double().cpu().numpy()
        sees = np.arange(kv[0] - new[0], kv[0]) >= p
        assert np.isnan(got[sees]).all() and np.isnan(lse.cpu().numpy()[sees]).all()
        assert (np.abs(got - want[0]) <= 2.0 ** -7 * want[2] + 2.0 ** -8 * np.abs(want[0]) + 1e-6)[~sees].all()


def test_scores_of_any_size_and_sign(ops):
    """Large scores (one key takes all), a negative and a zero scale."""
    for new, kv in (([2], [50]), ([40], [90])):
        b = Batch(new, kv, 4, 2, 64, 16, seed=4)
        for scale in (30.0, -0.125, 1e-30):
            verify(ops, b, f"scale {scale} new={new}", scale=scale)
