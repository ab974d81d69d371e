"""paged_attention with a block table wider than its sequences (the capacity that a captured program keeps), and batches
with as many row tiles as they can have: sequences of just more rows than the kernel for few rows takes."""
import numpy as np
import pytest

from attention_helpers import Batch, attend, check
from gpu_helpers import announce
from oracle import attention as oracle

pytestmark = pytest.mark.gpu


def widen(b, width, entry):
    table = np.full((b.B, width), entry, np.int32)
    table[:, :b.width] = b.table
    b.table, b.width = table, width


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("new", [[17] * 40, [17, 1] * 20, [33] * 12 + [1] * 30, [1] * 30 + [129, 16, 17, 15, 128, 0, 130]])
def test_most_row_tiles(new, fmt):
    """Key heads of one query head each, so that a token is a row; 16 rows are few, because the table is wide."""
    from weight_only_quantized_w4a16_amd import ops
    rng = np.random.default_rng(len(new))
    kv = [n + int(rng.integers(0, 60)) for n in new]
    b = Batch(new, kv, 8, 8, 64, 16, fmt, seed=len(new), extra_tokens=1)
    want = oracle.paged_attention(b.q, b.k, b.v, b.table, b.q_offsets, b.kv_len, 0.125)
    for width, entry in ((b.width, -1), (4096, -1), (4096, 0)):
        widen(b, width, entry)
        for m in (0, max(new)):
            announce(f"{new[:3]}.. {fmt} table of {width} max_q={m}")
            out, lse = attend(ops, b, max_q=m)
            check(b, out, lse, want, f"table of {width} max_q={m}")


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("new,window,sinks", [([1, 1, 1], 0, 0), ([4, 1, 3], 0, 0), ([1, 1, 1], 40, 3), ([70, 20, 1], 0, 0), ([70, 20, 1], 40, 3)])
def test_wide_tables(new, window, sinks, fmt):
    """Tables of 65536 positions behind sequences of hundreds: the plan sees the width, the result does not."""
    from weight_only_quantized_w4a16_amd import ops
    for D, Hq, Hkv in ((128, 8, 2), (64, 6, 3)):
        b = Batch(new, [300, 77, 190], Hq, Hkv, D, 16, fmt, seed=D)
        want = oracle.paged_attention(b.q, b.k, b.v, b.table, b.q_offsets, b.kv_len, D ** -0.5, window, sinks)
        widen(b, 4096, b.pages - 1)                      # a page that is there: positions past the end, not missing pages
        for m in (0, max(new)):
            announce(f"wide table {new} {fmt} D={D} window={window} max_q={m}")
            out, lse = attend(ops, b, window=window, sinks=sinks, max_q=m)
            check(b, out, lse, want, f"D={D} max_q={m}")


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_wide_table_behind_a_shared_prefix(fmt):
    from weight_only_quantized_w4a16_amd import ops
    prefix, Hkv, D = 2048, 8, 128
    new = [1, 17, 3, 18, 1, 17, 2, 40, 1]
    kv = [prefix + n + 9 * i for i, n in enumerate(new)]
    b = Batch(new, kv, Hkv, Hkv, D, 64, fmt, seed=5, shared=prefix)
    want = oracle.paged_attention(b.q, b.k, b.v, b.table, b.q_offsets, b.kv_len, D ** -0.5)
    for width in (b.width, 1024):
        widen(b, width, -1)
        for m in (0, 40):
            announce(f"shared, table of {width} {fmt} max_q={m}")
            out, lse = attend(ops, b, shared=prefix, max_q=m)
            check(b, out, lse, want, f"table of {width} max_q={m}")
