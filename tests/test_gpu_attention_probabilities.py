"""What sequences of few rows lose to the rounding of their probabilities: nothing, they enter the product with the values
as two bf16 numbers.  The bound is one that a single rounding to bf16 does not meet (shown on the CPU with the oracle)."""
import numpy as np
import pytest

from attention_helpers import Batch
from gpu_helpers import announce
from oracle import attention as oracle


def bounds(b, want):
    """As in attention_helpers.check, but for the probabilities: as the sum of two bf16 numbers each is off by half a step of
    the second one, which is no larger than half a step of the first: 2^-8 2^-8 of it."""
    y, l64, mean, reach = want
    n = int(b.kv_len.max())
    x = (2 * (b.D + 4) + 8) * 2.0 ** -24 * reach
    rel = np.expm1(2 * x) + 2.0 ** -16 + 2.0 ** -20 + n * 2.0 ** -23
    return rel[..., None] * mean + 2.0 ** -8 * (1 + 2.0 ** -6) * np.abs(y) + 1e-30


# up to 16 rows (tokens and heads of a key head) a sequence
BATCHES = {"decode": ([1] * 6, [3, 5, 17, 40, 9, 130], 4, 2), "16 rows": ([4, 1, 2], [30, 7, 120], 8, 2),
           "a sequence": ([2], [25], 16, 2), "a wide group": ([1, 1], [12, 33], 32, 2)}


def case(name, D, fmt):
    new, kv, Hq, Hkv = BATCHES[name]
    b = Batch(new, kv, Hq, Hkv, D, 16, fmt, seed=D + len(new))
    return b, new


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("name", BATCHES)
def test_few_rows_round_no_probabilities(name, D, fmt):
    from attention_helpers import attend
    from weight_only_quantized_w4a16_amd import ops
    b, new = case(name, D, fmt)
    want = oracle.paged_attention(b.q, b.k, b.v, b.table, b.q_offsets, b.kv_len, D ** -0.5)
    for m in (0, max(new)):
        announce(f"probabilities {name} {fmt} D={D} max_q={m}")
        out, _ = attend(ops, b, max_q=m)
        err = np.abs(out.double().cpu().numpy() - want[0])
        assert (err <= bounds(b, want)).all(), float((err / bounds(b, want)).max())


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("name", BATCHES)
def test_the_bound_tells_a_rounded_probability(name, fmt, monkeypatch):
    """The oracle with probabilities of one bf16 number misses the bound in every batch."""
    import torch
    b, _ = case(name, 64, fmt)
    want = oracle.paged_attention(b.q, b.k, b.v, b.table, b.q_offsets, b.kv_len, 0.125)
    exp = np.exp
    monkeypatch.setattr(oracle.np, "exp", lambda x: torch.from_numpy(exp(x)).to(torch.bfloat16).double().numpy())
    planted = oracle.paged_attention(b.q, b.k, b.v, b.table, b.q_offsets, b.kv_len, 0.125)[0]
    monkeypatch.undo()
    rounded = torch.from_numpy(planted).to(torch.bfloat16).double().numpy()
    assert (np.abs(rounded - want[0]) > bounds(b, want)).any()
