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
