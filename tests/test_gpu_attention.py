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


def verify(ops, b, what, scale=None, window=0, sinks=0, shared=0, max_q=0):
    announce(what)
    out, lse = attend(ops, b, scale, window, sinks, shared, max_q)
    want = oracle.paged_attention(b.q, b.k, b.v, b.table, b.q_offsets, b.kv_len, scale or b.D ** -0.5, window, sinks)
    return check(b, out, lse, want, what)


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
