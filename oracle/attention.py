"""CPU oracle of the operators between the qkv product and the o product, in fp64
(test infrastructure only): the norm and rotation of query and key heads, the
append to a paged cache, and causal attention over it with a sliding window and
first positions that stay visible.

Inputs are float64 arrays of the values the library receives, lists are numpy
integers.
"""
import numpy as np


def norm_rope(x, weight, eps, positions, inv_freq, rotary_dim, interleaved):
    """x [T, H, D] -> normed per head (weight None: not) and rotated by the positions' angles."""
    x = x.astype(np.float64)
    if weight is not None:
        x = x / np.sqrt(np.mean(x * x, axis=-1, keepdims=True) + eps) * weight
    out = x.copy()
    half = rotary_dim // 2
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        angle = positions.astype(np.float64) * inv_freq[i]
        c, s = np.cos(angle)[:, None], np.sin(angle)[:, None]
        out[..., a] = x[..., a] * c - x[..., b] * s
        out[..., b] = x[..., b] * c + x[..., a] * s
    return out


def places(T, q_offsets, kv_len):
    """(sequence, position) of every token; sequence -1 for tokens of none."""
    seq, pos = np.full(T, -1), np.zeros(T, np.int64)
    for b in range(len(kv_len)):
        lo, hi = q_offsets[b], q_offsets[b + 1]
        for t in range(lo, hi):
            seq[t], pos[t] = b, max(int(kv_len[b]), 0) - (hi - lo) + (t - lo)
    return seq, pos


def cache_rows(table_row, length, pages, page_size):
    """(position, page, slot) of the positions below `length` that have a page."""
    out = []
    for j in range(min(max(int(length), 0), len(table_row) * page_size)):
        p = int(table_row[j // page_size])
        if 0 <= p < pages:
            out.append((j, p, j % page_size))
    return out


def paged_attention(q, k, v, table, q_offsets, kv_len, scale, window=0, sinks=0):
    """q [T, Hq, D]; k, v [pages, Hkv, page, D].  Returns out [T, Hq, D], lse [T, Hq] and, for tolerances, the softmax's
    mean of |v| and the largest sum of |scale q_i k_i| over the keys a row sees (rows of no sequence: NaN)."""
    T, Hq, D = q.shape
    pages, Hkv, page, _ = k.shape
    G = Hq // Hkv
    out, mean = np.full((T, Hq, D), np.nan), np.full((T, Hq, D), np.nan)
    lse, reach = np.full((T, Hq), np.nan), np.zeros((T, Hq))
    for b in range(len(kv_len)):
        rows = cache_rows(table[b], kv_len[b], pages, page)
        at = np.array([r[0] for r in rows], np.int64)
        pg, sl = np.array([r[1] for r in rows], np.int64), np.array([r[2] for r in rows], np.int64)
        lo, hi = q_offsets[b], q_offsets[b + 1]
        for t in range(lo, hi):
            pos = max(int(kv_len[b]), 0) - (hi - lo) + (t - lo)
            sees = at <= pos
            if window:
                sees &= (at > pos - window) | (at < sinks)
            for h in range(Hq):
                kk, vv = k[pg[sees], h // G, sl[sees]], v[pg[sees], h // G, sl[sees]]
                with np.errstate(all="ignore"):
                    s = kk @ q[t, h] * scale if len(kk) else np.zeros(0)
                    if len(s) == 0 or np.all(s == -np.inf):
                        out[t, h], mean[t, h], lse[t, h] = 0, 0, -np.inf
                        continue
                    m = np.max(s)
                    p = np.exp(s - m)
                    out[t, h], mean[t, h] = p @ vv / p.sum(), p @ np.abs(vv) / p.sum()
                    lse[t, h] = m + np.log(p.sum())
                    reach[t, h] = np.max(np.abs(kk) @ np.abs(q[t, h])) * abs(scale)
    return out, lse, mean, reach
