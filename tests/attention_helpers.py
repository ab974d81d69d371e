"""Batches and caches for the attention tests, made on the CPU from a seed, and the tolerance of attention's outputs."""
import numpy as np
import torch

from oracle import fp8_e4m3 as f8


def bf16(x):
    """float64 values rounded to bf16, and the tensor that holds them."""
    t = torch.from_numpy(np.ascontiguousarray(x)).to(torch.bfloat16)
    return t.to(torch.float64).numpy(), t


class Batch:
    """Sequences of `new` tokens and `kv` positions over a paged cache; unused rows hold `junk`."""

    def __init__(self, new, kv, Hq, Hkv, D, page, fmt="bf16", seed=0, extra_tokens=0, junk=float("nan"), shared=0, spare=2):
        rng = np.random.default_rng(seed)
        self.Hq, self.Hkv, self.D, self.page, self.fmt = Hq, Hkv, D, page, fmt
        self.B, self.T = len(new), sum(new) + extra_tokens
        self.q_offsets = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        self.kv_len = np.array(kv, np.int32)
        first = shared // page
        need = [max(0, -(-k // page) - first) for k in kv]
        self.width = max(1, first + max(need, default=0))
        self.pages = first + sum(need) + spare
        order = rng.permutation(self.pages)
        self.table = np.full((self.B, self.width), -1, np.int32)
        self.table[:, :first] = order[:first]
        at = first
        for b, n in enumerate(need):
            self.table[b, first:first + n] = order[at:at + n]
            at += n
        self.q, self.q_t = bf16(rng.standard_normal((self.T, Hq, D)) * 1.5)
        used = np.zeros((self.pages, page), bool)
        for b in range(self.B):
            for j in range(max(int(kv[b]), 0)):
                used[self.table[b, j // page], j % page] = True
        used = np.broadcast_to(used[:, None, :], (self.pages, Hkv, page))
        gain = np.exp(0.3 * rng.standard_normal(D))
        for name in ("k", "v"):
            x = rng.standard_normal((self.pages, Hkv, page, D)) * gain
            if fmt == "bf16":
                x[~used] = junk
                values, t = bf16(x)
                scale_t = None
            else:
                s = (np.abs(x).max(-1) / 448).astype(np.float32)
                codes = f8.e4m3_encode((x / s[..., None]).astype(np.float32))
                codes[~used] = 0x7f if np.isnan(junk) else 0x7e
                s[~used] = junk
                with np.errstate(invalid="ignore"):
                    values = f8.e4m3_decode(codes).astype(np.float64) * s[..., None].astype(np.float64)
                t, scale_t = torch.from_numpy(codes.view(np.uint8)), torch.from_numpy(s)
            setattr(self, name, values)
            setattr(self, name + "_t", t)
            setattr(self, name + "_scale_t", scale_t)

    def device(self):
        """The tensors on the GPU, by name."""
        to = lambda t: None if t is None else t.cuda()
        d = {n: to(getattr(self, n + "_t")) for n in ("q", "k", "v", "k_scale", "v_scale")}
        for n in ("q_offsets", "kv_len", "table"):
            d[n] = torch.from_numpy(getattr(self, n)).cuda()
        return d


def attend(ops, b, scale=None, window=0, sinks=0, shared=0, max_q=0, lse=True, d=None, fill=7.0):
    """paged_attention of a batch: (out, lse) tensors; rows that the call does not write keep `fill`."""
    d = d or b.device()
    out = torch.full((b.T, b.Hq, b.D), fill, dtype=torch.bfloat16, device="cuda")
    stat = torch.full((b.T, b.Hq), fill, dtype=torch.float32, device="cuda") if lse else None
    need = ops.paged_attention_workspace_bytes(b.T, b.B, b.width, b.Hq, b.Hkv, b.D, b.page, shared, max_q)
    ws = torch.zeros(need, dtype=torch.uint8, device="cuda") if need else None
    ops.paged_attention(d["q"], d["k"], d["v"], d["k_scale"], d["v_scale"], b.pages, b.page, d["q_offsets"], d["kv_len"],
                        d["table"], b.T, b.B, b.width, b.Hq, b.Hkv, b.D, scale or b.D ** -0.5, window, sinks, shared, max_q, out,
                        stat, ws, need)
    if ws is not None:
        torch.cuda.synchronize()
        assert not ws[:65536].any(), "completion counters left behind"
    return out, stat


def check(b, out, lse, want, what=""):
    """The outputs against the oracle's (out, lse, mean |v|, reach).

    A score is a sum of D products of bf16 (or e4m3 times scale) numbers in fp32 and two products: off by at most
    (D + 4) 2^-24 of the sum of magnitudes, `reach`; so is its exponent's reference.  A probability is off by e^2x - 1 with
    x = 2 (D + 4) 2^-24 reach, by the hardware's exponential (2^-22), by what fp32 exponents lose (|s| 2^-24 of base-2 scores
    up to 2 reach), and by the rounding to bf16, 2^-8; the sums over n keys are off by n 2^-24 at most, and each joining of
    chunks by a few 2^-24.  All of it is relative to the mean of |v|; the output's rounding, 2^-8, to the output."""
    y, l64, mean, reach = want
    live = ~np.isnan(mean).any(-1) | ~np.isnan(l64)
    n = max(1, int(b.kv_len.max(initial=0)))
    x = (2 * (b.D + 4) + 8) * 2.0 ** -24 * reach
    rel = np.expm1(2 * x) + 2.0 ** -8 + 2.0 ** -20 + n * 2.0 ** -23
    got = out.double().cpu().numpy()
    bound = rel[..., None] * mean + 2.0 ** -8 * (1 + 2.0 ** -6) * np.abs(y) + 1e-30
    with np.errstate(invalid="ignore"):
        err = np.abs(got - y)
    ok = err <= bound
    assert ok[live].all(), f"{what}: {np.argwhere(~ok & live[..., None])[:4]} worst {np.nanmax((err / bound)[live])}"
    assert (got[~live] == 7.0).all(), f"{what}: rows of no sequence were written"
    if lse is not None:
        g = lse.double().cpu().numpy()
        empty = live & (l64 == -np.inf)
        assert (g[empty] == -np.inf).all(), what
        full = live & ~empty
        lb = 2 * x + 2.0 ** -20 + n * 2.0 ** -23 + 2.0 ** -22 * np.abs(np.where(full, l64, 0))
        with np.errstate(invalid="ignore"):
            assert (np.abs(g - l64) <= lb)[full].all(), f"{what}: lse"
        assert (g[~live] == 7.0).all(), what
    return float(np.nanmax((err / bound)[live])) if live.any() else 0.0
