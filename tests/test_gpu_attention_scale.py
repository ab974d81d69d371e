"""paged_attention with a scale of zero: every key that a row sees counts alike, whichever kernel takes the row; and scales
that leave every score as good as zero."""
import numpy as np
import pytest
import torch

from attention_helpers import Batch, check
from gpu_helpers import announce
from oracle import attention as oracle

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ops():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    from weight_only_quantized_w4a16_amd import ops as _ops
    return _ops


def attend(ops, b, scale, window=0, sinks=0, shared=0, max_q=0):
    d = b.device()
    out = torch.full((b.T, b.Hq, b.D), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((b.T, b.Hq), 7.0, dtype=torch.float32, device="cuda")
    need = ops.paged_attention_workspace_bytes(b.T, b.B, b.width, b.Hq, b.Hkv, b.D, b.page, shared, max_q)
    ws = torch.zeros(need, dtype=torch.uint8, device="cuda") if need else None
    ops.paged_attention(d["q"], d["k"], d["v"], d["k_scale"], d["v_scale"], b.pages, b.page, d["q_offsets"], d["kv_len"], d["table"],
                        b.T, b.B, b.width, b.Hq, b.Hkv, b.D, scale, window, sinks, shared, max_q, out, lse, ws, need)
    return out, lse


SCALES = [0.0, -0.0, 1e-45, -1e-40]


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("window,sinks", [(0, 0), (40, 3)])
@pytest.mark.parametrize("new,kv", [([2], [50]), ([70], [200]), ([33, 1, 0, 90], [40, 600, 70, 1100])])
def test_scale_zero(ops, new, kv, window, sinks, D, fmt):
    b = Batch(new, kv, 4, 2, D, 16, fmt, seed=D + len(kv), extra_tokens=1)
    for scale in SCALES:
        want = oracle.paged_attention(b.q, b.k, b.v, b.table, b.q_offsets, b.kv_len, scale, window, sinks)
        for m in (0, max(new)):
            what = f"scale {scale} {new} {kv} window {window} {fmt} D={D} max_q={m}"
            announce(what)
            check(b, *attend(ops, b, scale, window, sinks, 0, m), want, what)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_scale_zero_behind_a_shared_prefix(ops, fmt):
    prefix, D, Hkv = 2048, 128, 8
    assert 8 * prefix * Hkv * D * 4 >= 64 << 20          # a pass of its own
    new = [1, 1, 1, 3, 1, 1, 1, 40, 1]
    kv = [prefix + m for m in (1, 300, 2, 17, 64, 129, 5, 40, 1)]
    kv[2] = prefix - 7                                   # new tokens inside the prefix: masked positions there too
    b = Batch(new, kv, Hkv, Hkv, D, 64, fmt, seed=3, shared=prefix)
    want = oracle.paged_attention(b.q, b.k, b.v, b.table, b.q_offsets, b.kv_len, 0.0)
    for m in (0, 40):
        announce(f"scale 0 shared {fmt} max_q={m}")
        check(b, *attend(ops, b, 0.0, 0, 0, prefix, m), want, f"{fmt} max_q={m}")


@pytest.mark.parametrize("new,kv", [([3], [40]), ([80], [140])])
def test_scale_zero_of_products_that_are_not_finite(ops, new, kv):
    """0 times an infinite or NaN product is NaN, in both kernels, for the rows that see it and for no others."""
    for name in ("key", "query"):
        b = Batch(new, kv, 2, 1, 64, 16, seed=2)
        n, p = new[0], kv[0] - 2
        sees = np.arange(kv[0] - n, kv[0]) >= p
        if name == "key":
            b.k_t[b.table[0, p // 16], :, p % 16, 5] = float("inf")
        else:
            sees = np.arange(n) == 1
            b.q_t[1, :, 9] = float("-inf")
        # the rows that see it by formula, the others as if it were not there
        clean = oracle.paged_attention(b.q, b.k, b.v, b.table, b.q_offsets, b.kv_len, 0.0)
        announce(f"scale 0, infinite {name} {new}")
        out, lse = attend(ops, b, 0.0)
        got = out.double().cpu().numpy()
        assert np.isnan(got[sees]).all() and np.isnan(lse.cpu().numpy()[sees]).all()
        assert (np.abs(got - clean[0]) <= 2.0 ** -7 * clean[2] + 2.0 ** -8 * np.abs(clean[0]) + 1e-6)[~sees].all()
