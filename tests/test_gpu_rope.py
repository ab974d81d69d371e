"""qk_norm_rope and kv_append against the oracle in 64 bits: norms, both pairings, partial rotation, far and negative
positions, ragged batches, positions without pages, extreme rows, and what must stay as it was."""
import numpy as np
import pytest
import torch

from attention_helpers import Batch, bf16
from gpu_helpers import announce
from oracle import attention as oracle
from oracle import fp8_e4m3 as f8

pytestmark = pytest.mark.gpu

EPS = 1e-6


@pytest.fixture(scope="module")
def ops():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    from weight_only_quantized_w4a16_amd import ops as _ops
    return _ops


def freqs(rot, base=500000.0):
    return base ** (-np.arange(rot // 2, dtype=np.float64) / max(rot // 2, 1))


def bound(want, x, weight, rot):
    """fp32 work before the one rounding: the norm's factor and weight (each product half a step, 2^-24; the reciprocal root
    2^-23), the hardware's sine and cosine (2^-22 absolute, the angle's turn rounded to 2^-25 of a turn: 2 pi 2^-25), on both
    elements of a pair; then half a step of bf16, 2^-8 of the value."""
    y = np.abs(x if weight is None else x / np.sqrt(np.mean(x * x, -1, keepdims=True) + EPS) * weight)
    pair = y.max(-1, keepdims=True) if rot else y
    return 2.0 ** -8 * (1 + 2.0 ** -7) * np.abs(want) + 2.0 ** -20 * (y + (pair if rot else 0)) + 1e-38


def run_dense(ops, x, xt, T, Hq, Hkv, D, wq, wk, positions, rot, inter):
    q = torch.full((T, Hq, D), 7.0, dtype=torch.bfloat16, device="cuda")
    k = torch.full((T, Hkv, D), 7.0, dtype=torch.bfloat16, device="cuda")
    f = torch.from_numpy(freqs(rot)).cuda() if rot else None
    ops.qk_norm_rope(xt.cuda(), wq and wq[1].cuda(), wk and wk[1].cuda(), EPS, torch.from_numpy(positions).cuda(), f, rot, inter,
                     T, Hq, Hkv, D, q, k)
    for name, got, lo, hi, w in (("q", q, 0, Hq, wq), ("k", k, Hq, Hq + Hkv, wk)):
        part = x.reshape(T, Hq + 2 * Hkv, D)[:, lo:hi]
        want = oracle.norm_rope(part, w and w[0], EPS, positions, freqs(rot), rot, inter)
        err = np.abs(got.double().cpu().numpy() - want)
        ok = err <= bound(want, part, w and w[0], rot)
        assert ok.all(), (name, np.argwhere(~ok)[:3])


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("D,rot", [(64, 0), (64, 16), (64, 64), (128, 32), (128, 80), (128, 128)])
def test_dense(ops, D, rot, inter):
    rng = np.random.default_rng(D + rot)
    for T, Hq, Hkv, norm in ((1, 4, 1, "both"), (7, 5, 5, "none"), (33, 6, 2, "q"), (300, 16, 2, "k")):
        announce(f"qk_norm_rope T={T} Hq={Hq} Hkv={Hkv} D={D} rot={rot} inter={inter} norm={norm}")
        x, xt = bf16(rng.standard_normal((T, (Hq + 2 * Hkv) * D)) * 3)
        w = [bf16(1 + 0.3 * rng.standard_normal(D)) for _ in range(2)]
        positions = rng.integers(-5, 200000, T).astype(np.int32)
        positions[0] = 2 ** 31 - 1 if T > 1 else 0
        run_dense(ops, x, xt, T, Hq, Hkv, D, w[0] if norm in ("both", "q") else None, w[1] if norm in ("both", "k") else None,
                  positions, rot, inter)


def test_far_positions(ops):
    """Every position up to 2^31 keeps its angle to fp64's accuracy: a one in the first half turns into (cos, sin)."""
    T, D = 2000, 128
    rng = np.random.default_rng(3)
    positions = rng.integers(2 ** 30, 2 ** 31, T).astype(np.int32)
    x = np.zeros((T, 3 * D))
    x[:, :D // 2] = 1.0
    x, xt = bf16(x)
    run_dense(ops, x, xt, T, 1, 1, D, None, None, positions, D, False)


@pytest.mark.parametrize("size", [1e-30, 1e30])
def test_norm_of_extreme_rows(ops, size):
    """The squares neither overflow nor vanish (eps 1e-6 dominates the small rows)."""
    rng = np.random.default_rng(4)
    x, xt = bf16(rng.standard_normal((9, 4 * 64)) * size)
    w = bf16(1 + 0.3 * rng.standard_normal(64))
    run_dense(ops, x, xt, 9, 2, 1, 64, w, w, np.arange(9, dtype=np.int32), 64, False)


def append(ops, b, x_t, wq, wk, rot, inter, d, fill=7.0):
    q = torch.full((b.T, b.Hq, b.D), fill, dtype=torch.bfloat16, device="cuda")
    f = torch.from_numpy(freqs(rot)).cuda() if rot else None
    ops.kv_append(x_t.cuda(), wq and wq[1].cuda(), wk and wk[1].cuda(), EPS, f, rot, inter, d["q_offsets"], d["kv_len"], d["table"],
                  b.T, b.B, b.width, b.Hq, b.Hkv, b.D, d["k"], d["v"], d["k_scale"], d["v_scale"], b.pages, b.page, q)
    return q


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("D,rot,inter,norm", [(128, 128, False, True), (128, 64, True, False), (64, 64, False, True), (64, 0, False, False)])
def test_append(ops, fmt, D, rot, inter, norm):
    rng = np.random.default_rng(D + rot)
    for new, kv, Hq, Hkv, page in (([1], [1], 4, 2, 16), ([1, 0, 1, 3], [17, 5, 0, 2], 3, 1, 16), ([40, 5, 70], [41, 300, 70], 8, 8, 32)):
        b = Batch(new, kv, Hq, Hkv, D, page, fmt, seed=len(new), extra_tokens=2)
        announce(f"kv_append {new} {kv} Hq={Hq} Hkv={Hkv} D={D} page={page} {fmt} rot={rot} inter={inter} norm={norm}")
        if len(new) == 3:
            b.table[1, 9] = -1                       # positions 288 .. 299 of the second sequence have no page
            b.table[2, 1] = b.pages
        x, xt = bf16(rng.standard_normal((b.T, (Hq + 2 * Hkv) * D)) * 2)
        wq, wk = (bf16(1 + 0.3 * rng.standard_normal(D)) for _ in range(2)) if norm else (None, None)
        d = b.device()
        before = {n: d[n].clone() for n in ("k", "v", "k_scale", "v_scale") if d[n] is not None}
        q = append(ops, b, xt, wq, wk, rot, inter, d)
        seq, pos = oracle.places(b.T, b.q_offsets, b.kv_len)
        heads = x.reshape(b.T, Hq + 2 * Hkv, D)
        live = seq >= 0
        want = oracle.norm_rope(heads[:, :Hq], wq and wq[0], EPS, pos, freqs(rot), rot, inter)
        got = q.double().cpu().numpy()
        assert (np.abs(got - want) <= bound(want, heads[:, :Hq], wq and wq[0], rot))[live].all()
        assert (got[~live] == 7.0).all(), "queries of no sequence were written"
        key = oracle.norm_rope(heads[:, Hq:Hq + Hkv], wk and wk[0], EPS, pos, freqs(rot), rot, inter)
        for name, val, src, w, r in (("k", key, heads[:, Hq:Hq + Hkv], wk, rot), ("v", heads[:, Hq + Hkv:], heads[:, Hq + Hkv:], None, 0)):
            slack = bound(val, src, w and w[0], r)
            got = d[name].cpu()
            untouched = np.ones((b.pages, page), bool)
            for t in range(b.T):
                if not live[t] or not 0 <= pos[t] < b.width * page:
                    continue
                p = b.table[seq[t], pos[t] // page]
                if not 0 <= p < b.pages:
                    continue
                untouched[p, pos[t] % page] = False
                row = got[p, :, pos[t] % page]
                if fmt == "bf16":
                    assert (np.abs(row.double().numpy() - val[t]) <= slack[t]).all(), (name, t)
                else:
                    s = d[name + "_scale"].cpu()[p, :, pos[t] % page].double().numpy()[:, None]
                    top = np.abs(val[t]).max(-1, keepdims=True)
                    fp32 = slack[t] - 2.0 ** -8 * (1 + 2.0 ** -7) * np.abs(val[t])      # the work before the code
                    assert (np.abs(s * 448 - top) <= fp32.max(-1, keepdims=True) + 2.0 ** -22 * top).all(), (name, t)
                    value = f8.e4m3_decode(row.numpy()).astype(np.float64) * s
                    # half a step of e4m3, 2^-4 of a normal value, 2^-10 scales of a subnormal one
                    near = 2.0 ** -4 * (1 + 2.0 ** -10) * np.abs(val[t]) + 2.0 ** -10 * s * 1.001 + 2 * fp32
                    assert (np.abs(value - val[t]) <= near).all(), (name, t)
            same = torch.from_numpy(untouched)[:, None, :].expand(-1, Hkv, -1)
            for n in (name, name + "_scale"):
                if d[n] is not None:
                    bits = lambda z: z.cpu().contiguous().view(torch.int32 if z.dtype == torch.float32 else torch.int16 if z.dtype == torch.bfloat16 else torch.uint8)
                    assert torch.equal(bits(d[n])[same], bits(before[n])[same]), f"{n}: rows of other positions changed"


def test_append_rows_with_nan_and_zeros(ops):
    """8-bit rows: zeros get scale 0 and codes 0; a NaN or an infinity shows in the scale."""
    b = Batch([4], [4], 1, 1, 64, 16, "e4m3")
    x = np.ones((4, 3 * 64))
    x[0, 64:] = 0
    x[1, 64 + 5], x[2, 128 + 9], x[3, 128:] = np.nan, np.inf, 0
    d = b.device()
    append(ops, b, bf16(x)[1], None, None, 0, False, d)
    p = int(b.table[0, 0])
    ks, vs = d["k_scale"][p, 0, :4].cpu(), d["v_scale"][p, 0, :4].cpu()
    assert ks[0] == 0 and vs[0] == 0 and vs[3] == 0 and (d["k"][p, 0, 0] == 0).all() and (d["v"][p, 0, 3] == 0).all()
    assert torch.isnan(ks[1]) and torch.isinf(vs[2]) and ks[3] == np.float32(1) / np.float32(448)
