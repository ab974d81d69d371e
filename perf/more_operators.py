"""Cases of the attention half of a decoder block, from the fused qkv product's output to the o product's input.

  norm_rope  q and k of a fused qkv row: RMS norm of every head and rotation by position, in one pass
  append     the same for q, while k and v go into a paged cache (bf16, or e4m3 codes with a scale per token and head)
  attend     causal attention of the new tokens over the paged cache, with a sliding window and first tokens that stay visible
  shared     the same for a batch whose sequences begin with the same pages, which are read once for all

`own` chooses between the plain torch form of each operator and the library's entry points.  Head layouts are those of the
repository's dense and expert layers (32 or 64 query heads over 8 or 4 key heads of 128) and heads of 64; batches and
lengths run from one token to the thousands of a prefill over caches of tens of thousands of tokens.
"""
import math
import random

import torch

own = False

DEV = "cuda"
EPS = 1e-6
BASE = 500000.0


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one decode token of a model with query and key norms
        {"name": "norm rope 1", "op": "norm_rope", "T": 1, "Hq": 32, "Hkv": 4, "D": 128, "norm": True, "rot": 128, "inter": False},
        # a prefill chunk of a wide model; an odd number of tokens
        {"name": "norm rope 8191", "op": "norm_rope", "T": 8191, "Hq": 64, "Hkv": 8, "D": 128, "norm": True, "rot": 128,
         "inter": False},
        # the largest decode batch, a token each into a bf16 cache
        {"name": "append 16 bf16", "op": "append", "B": 16, "n": 1, "ragged": False, "kv": 8192, "Hq": 32, "Hkv": 8, "D": 128,
         "page": 16, "fmt": "bf16", "norm": False, "rot": 128, "inter": False},
        # the prefill chunks of a few sequences into an 8-bit cache
        {"name": "append 5 x 1500 e4m3", "op": "append", "B": 5, "n": 1500, "ragged": True, "kv": 4000, "Hq": 32, "Hkv": 4,
         "D": 128, "page": 64, "fmt": "e4m3", "norm": True, "rot": 128, "inter": False},
        # one sequence's decode step: latency, and one long axis to split
        {"name": "decode 1 x 16384 bf16", "op": "attend", "B": 1, "n": 1, "ragged": False, "kv": 16384, "Hq": 32, "Hkv": 8,
         "D": 128, "page": 16, "fmt": "bf16", "window": 0, "sinks": 0, "lse": False},
        # a large batch of sequences of all lengths over an 8-bit cache
        {"name": "decode 64 ragged e4m3", "op": "attend", "B": 64, "n": 1, "ragged": True, "kv": 8192, "Hq": 32, "Hkv": 8,
         "D": 128, "page": 64, "fmt": "e4m3", "window": 0, "sinks": 0, "lse": False},
        # long conversations under a sliding window, the first tokens kept
        {"name": "decode 16 window bf16", "op": "attend", "B": 16, "n": 1, "ragged": True, "kv": 32768, "Hq": 64, "Hkv": 8,
         "D": 128, "page": 64, "fmt": "bf16", "window": 1024, "sinks": 4, "lse": False},
        # a prefill chunk behind as many tokens again
        {"name": "prefill 4096 of 8192 bf16", "op": "attend", "B": 1, "n": 4096, "ragged": False, "kv": 8192, "Hq": 32,
         "Hkv": 8, "D": 128, "page": 64, "fmt": "bf16", "window": 0, "sinks": 0, "lse": False},
        # prefill chunks of odd lengths, heads of 64 under a window, 8-bit cache; the statistics for a later merge
        {"name": "prefill 7 window e4m3", "op": "attend", "B": 7, "n": 1100, "ragged": True, "kv": 4500, "Hq": 32, "Hkv": 8,
         "D": 64, "page": 16, "fmt": "e4m3", "window": 512, "sinks": 4, "lse": True},
        # a few proposed tokens each, checked for three sequences behind one instruction
        {"name": "shared 3 x 4 of 1024 e4m3", "op": "shared", "B": 3, "n": 4, "ragged": False, "prefix": 1024, "kv": 1200,
         "Hq": 32, "Hkv": 4, "D": 128, "page": 16, "fmt": "e4m3", "lse": False},
        # a decode batch behind one long document
        {"name": "shared 32 of 8192 bf16", "op": "shared", "B": 32, "n": 1, "ragged": True, "prefix": 8192, "kv": 8704, "Hq": 32,
         "Hkv": 8, "D": 128, "page": 64, "fmt": "bf16", "lse": False},
        # a large decode batch behind a longer one, 8-bit cache
        {"name": "shared 128 of 16384 e4m3", "op": "shared", "B": 128, "n": 1, "ragged": True, "prefix": 16384, "kv": 17200,
         "Hq": 64, "Hkv": 8, "D": 128, "page": 64, "fmt": "e4m3", "lse": False},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))))


HEADS = [(32, 8), (32, 4), (64, 8), (16, 16), (8, 1), (24, 8), (10, 2)]


def draw(rng):
    op = rng.choice(["norm_rope", "append", "attend", "attend", "attend", "shared"])
    Hq, Hkv = rng.choice(HEADS)
    D = rng.choice([64, 128, 128])
    case = {"op": op, "Hq": Hq, "Hkv": Hkv, "D": D}
    if op in ("norm_rope", "append"):
        case.update(norm=rng.random() < 0.6, rot=rng.choice([D, D, D // 2]), inter=rng.random() < 0.3)
    if op == "norm_rope":
        case["T"] = _log(rng, 1, 8191 * 72 // (Hq + Hkv))
        return case
    case.update(page=rng.choice([16, 32, 64, 128, 256]), fmt=rng.choice(["bf16", "e4m3"]), ragged=rng.random() < 0.7)
    if op == "append":
        case["B"] = _log(rng, 1, 64)
        case["n"] = rng.choice([1, _log(rng, 1, 8192 // case["B"])])
        case["kv"] = case["n"] + _log(rng, 1, 4096)
        return case
    case["lse"] = rng.random() < 0.3
    if op == "shared":
        case["B"] = _log(rng, 2, 128)
        case["n"] = rng.choice([1, 1, rng.randint(2, 8)])
        case["prefix"] = 256 * _log(rng, 1, min(64, max(1, (1 << 21) // (case["B"] * case["n"] * Hq))))
        case["kv"] = case["prefix"] + case["n"] + _log(rng, 1, 800)
        return case
    if rng.random() < 0.5:
        # decode: the whole cache is read
        case["n"] = rng.choice([1, 1, 1, rng.randint(2, 6)])
        case["B"] = _log(rng, 1, 64)
        case["kv"] = case["n"] + _log(rng, 1, min(32768, (1 << 28) // (case["B"] * Hkv * D)))
    else:
        # prefill: n new tokens each behind up to as many again, or more
        case["B"] = _log(rng, 1, 8)
        case["n"] = _log(rng, 17, 4096 // case["B"])
        case["kv"] = case["n"] + _log(rng, 1, min(4096, (1 << 30) // (case["B"] * case["n"] * Hq) - case["n"] // 2))
    windowed = rng.random() < 0.4
    case["window"] = _log(rng, 1, 4096) if windowed else 0
    case["sinks"] = rng.choice([0, 1, 4, 37]) if windowed else 0
    return case


# ------------------------------------------------------------------ inputs

def _lengths(case):
    """New tokens and keys (new ones included) of every sequence; the first one has the case's full lengths."""
    B, n, kv, least = case["B"], case["n"], case["kv"], case.get("prefix", 0)
    if not case["ragged"]:
        return [n] * B, [kv] * B
    rng = random.Random("%d %d %d" % (B, n, kv))
    new = [n] + [rng.randint(max(1, n // 4), n) for _ in range(B - 1)]
    return new, [kv] + [rng.randint(least + m, kv) for m in new[1:]]


def _cache(g, case, pages):
    """Keys and values as earlier appends left them: normal values with a few larger channels."""
    shape = (pages, case["Hkv"], case["page"], case["D"])
    out = {}
    for name in ("k", "v"):
        x = torch.randn(shape, generator=g, device=DEV)
        x *= torch.exp(0.3 * torch.randn(case["D"], generator=g, device=DEV))
        if case["fmt"] == "e4m3":
            s = x.abs().amax(3).clamp_min(1e-6) / 448.0
            out[name] = (x / s[..., None]).clamp_(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
            out[name + "_scale"] = s
        else:
            out[name], out[name + "_scale"] = x.to(torch.bfloat16), None
    return out


def _projected(g, T, case):
    """Rows of a fused qkv product: query, key and value heads side by side."""
    width = (case["Hq"] + 2 * case["Hkv"]) * case["D"]
    gain = torch.exp(0.4 * torch.randn(width, generator=g, device=DEV))
    return (torch.randn((T, width), generator=g, device=DEV) * gain).to(torch.bfloat16)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    st = dict(case)
    op, Hq, Hkv, D = case["op"], case["Hq"], case["Hkv"], case["D"]
    bf16 = dict(dtype=torch.bfloat16, device=DEV)
    if op == "norm_rope":
        T = case["T"]
        st["positions"] = torch.randint(0, 131072, (T,), generator=g, device=DEV, dtype=torch.int32)
        st["k_out"] = torch.empty((T, Hkv, D), **bf16)
    else:
        new, kv = _lengths(case)
        B, page, prefix, T = case["B"], case["page"], case.get("prefix", 0), sum(new)
        # pages in no order, the shared ones the same in every row; entries past a sequence's end are -1
        need = torch.tensor([(n - prefix + page - 1) // page for n in kv])
        own_pages = int(need.sum())
        width, first = (max(kv) + page - 1) // page, prefix // page
        order = torch.randperm(first + own_pages + 3, generator=g, device=DEV).to(torch.int32)
        table = torch.full((B, width), -1, dtype=torch.int32, device=DEV)
        table[:, :first] = order[:first]
        used = (torch.arange(width - first)[None, :] < need[:, None]).to(DEV)
        table[:, first:][used] = order[first:first + own_pages]
        st["table"], st["pages"], st["width"], st["T"] = table, first + own_pages + 3, width, T
        st["kv_len"] = torch.tensor(kv, dtype=torch.int32, device=DEV)
        st["q_offsets"] = torch.tensor([sum(new[:b]) for b in range(B + 1)], dtype=torch.int32, device=DEV)
        st["max_q"], st["max_kv"] = max(new), max(kv)
        st.update(_cache(g, case, st["pages"]))
    if op in ("norm_rope", "append"):
        st["qkv"] = _projected(g, T, case)
        half = case["rot"] // 2
        st["inv_freq"] = BASE ** (-torch.arange(half, dtype=torch.float64, device=DEV) / half)
        st["wq"], st["wk"] = (((1 + 0.2 * torch.randn(D, generator=g, device=DEV)).to(torch.bfloat16) if case["norm"] else None)
                              for _ in range(2))
        st["q_out"] = torch.empty((T, Hq, D), **bf16)
    else:
        st["q"] = torch.randn((T, Hq, D), generator=g, device=DEV).to(torch.bfloat16)
        st["scale"] = 1.0 / math.sqrt(D)
        st["out"] = torch.empty((T, Hq, D), **bf16)
        st["lse_out"] = torch.empty((T, Hq), dtype=torch.float32, device=DEV) if case["lse"] else None
        if own:
            from weight_only_quantized_w4a16_amd import ops
            st["ws_bytes"] = ops.paged_attention_workspace_bytes(T, st["B"], st["width"], Hq, Hkv, D, st["page"],
                                                                 st.get("prefix", 0), st["max_q"])
            st["ws"] = torch.zeros(st["ws_bytes"], dtype=torch.uint8, device=DEV) if st["ws_bytes"] else None
    return st


# ------------------------------------------------------------------ one pass

def run(state):
    return (_run_own if own else _run_plain)(state)


def _stored(st):
    """The cache whole: bf16, or e4m3 codes as the numbers they are beside their scales."""
    if st["fmt"] == "bf16":
        return {"k": st["k"], "v": st["v"]}
    return {"k": st["k"].view(torch.float8_e4m3fn), "v": st["v"].view(torch.float8_e4m3fn), "k_scale": st["k_scale"],
            "v_scale": st["v_scale"]}


def _run_own(st):
    from weight_only_quantized_w4a16_amd import ops
    Hq, Hkv, D = st["Hq"], st["Hkv"], st["D"]
    if st["op"] == "norm_rope":
        ops.qk_norm_rope(st["qkv"], st["wq"], st["wk"], EPS, st["positions"], st["inv_freq"], st["rot"], st["inter"], st["T"],
                         Hq, Hkv, D, st["q_out"], st["k_out"])
        return {"q": st["q_out"], "k": st["k_out"]}
    if st["op"] == "append":
        ops.kv_append(st["qkv"], st["wq"], st["wk"], EPS, st["inv_freq"], st["rot"], st["inter"], st["q_offsets"], st["kv_len"],
                      st["table"], st["T"], st["B"], st["width"], Hq, Hkv, D, st["k"], st["v"], st["k_scale"], st["v_scale"],
                      st["pages"], st["page"], st["q_out"])
        return {"q": st["q_out"], **_stored(st)}
    ops.paged_attention(st["q"], st["k"], st["v"], st["k_scale"], st["v_scale"], st["pages"], st["page"], st["q_offsets"],
                        st["kv_len"], st["table"], st["T"], st["B"], st["width"], Hq, Hkv, D, st["scale"], st.get("window", 0),
                        st.get("sinks", 0), st.get("prefix", 0), st["max_q"], st["out"], st["lse_out"], st["ws"], st["ws_bytes"])
    return _answer(st["out"], st["lse_out"])


def _answer(out, lse):
    return {"out": out} if lse is None else {"out": out, "lse": lse}


def _normed(x, w):
    x = x.float()
    if w is None:
        return x
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w.float()


def _rotated(st, x, positions):
    """x [T, H, D] turned by the positions' angles, pair by pair: (i, i + rot / 2), or (2 i, 2 i + 1)."""
    angle = positions.double()[:, None] * st["inv_freq"]
    cos, sin = torch.cos(angle).float()[:, None, :], torch.sin(angle).float()[:, None, :]
    rot, rest = x[..., :st["rot"]], x[..., st["rot"]:]
    if st["inter"]:
        a, b = rot[..., 0::2], rot[..., 1::2]
        return torch.cat((torch.stack((a * cos - b * sin, a * sin + b * cos), -1).flatten(-2), rest), -1)
    a, b = rot[..., :st["rot"] // 2], rot[..., st["rot"] // 2:]
    return torch.cat((a * cos - b * sin, a * sin + b * cos, rest), -1)


def _heads(st):
    Hq, Hkv = st["Hq"], st["Hkv"]
    x = st["qkv"].view(st["T"], Hq + 2 * Hkv, st["D"])
    return x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]


def _places(st):
    """The sequence and the position of every token."""
    t = torch.arange(st["T"], device=DEV)
    seq = torch.bucketize(t, st["q_offsets"].long(), right=True) - 1
    return seq, (st["kv_len"].long() - st["q_offsets"][1:].long())[seq] + t


def _store(st, name, x, page, slot):
    if st["fmt"] == "bf16":
        st[name][page, :, slot] = x.to(torch.bfloat16)
        return
    s = x.abs().amax(-1) / 448.0
    q = x / torch.where(s > 0, s, torch.ones_like(s))[..., None]
    st[name][page, :, slot] = q.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    st[name + "_scale"][page, :, slot] = s


def _fetched(st, name, page, slot):
    """Cached rows in 32 bits: [..., Hkv, D] for pages and slots of any shape."""
    x = st[name][page, :, slot]
    if st["fmt"] == "bf16":
        return x.float()
    return x.view(torch.float8_e4m3fn).float() * st[name + "_scale"][page, :, slot][..., None]


def _run_plain(st):
    if st["op"] in ("norm_rope", "append"):
        q, k, v = _heads(st)
        seq, positions = (None, st["positions"]) if st["op"] == "norm_rope" else _places(st)
        q = _rotated(st, _normed(q, st["wq"]), positions).to(torch.bfloat16)
        k = _rotated(st, _normed(k, st["wk"]), positions)
        if st["op"] == "norm_rope":
            return {"q": q, "k": k.to(torch.bfloat16)}
        page = st["table"][seq, positions // st["page"]].long()
        _store(st, "k", k, page, positions % st["page"])
        _store(st, "v", v.float(), page, positions % st["page"])
        return {"q": q, **_stored(st)}
    B, T, n, Hq, Hkv, D = (st[x] for x in ("B", "T", "max_q", "Hq", "Hkv", "D"))
    G = Hq // Hkv
    window, sinks, prefix = st.get("window", 0), st.get("sinks", 0), st.get("prefix", 0)
    kv = st["kv_len"].long()[:, None]
    seq, positions = _places(st)
    row = torch.arange(T, device=DEV) - st["q_offsets"].long()[seq]
    # every sequence's own keys: the first ones that stay visible, then the window's (all of them without one)
    if window:
        begin = (kv - n - window + 1).clamp_min(sinks)
        at = torch.cat((torch.arange(sinks, device=DEV).expand(B, sinks), begin + torch.arange(window + n - 1, device=DEV)), 1)
    else:
        at = (prefix + torch.arange(st["max_kv"] - prefix, device=DEV)).expand(B, st["max_kv"] - prefix)
    inside = at < kv
    page = st["table"].long().gather(1, torch.where(inside, at, torch.zeros_like(at)) // st["page"])
    kx, vx = (_fetched(st, name, page, at % st["page"]).permute(0, 2, 1, 3) for name in ("k", "v"))     # [B, Hkv, L, D]
    # queries padded to n a sequence, the heads of a group as rows of their key head
    q = torch.zeros((B, n, Hkv, G, D), device=DEV)
    q[seq, row] = st["q"].float().view(T, Hkv, G, D) * st["scale"]
    q = q.permute(0, 2, 1, 3, 4).reshape(B, Hkv, n * G, D)
    pos = torch.full((B, n), -1, dtype=torch.int64, device=DEV)
    pos[seq, row] = positions
    seen = inside[:, None, :] & (at[:, None, :] <= pos[:, :, None])
    if window:
        seen = seen & ((at[:, None, :] > pos[:, :, None] - window) | (at[:, None, :] < sinks))
    s = q @ kx.transpose(2, 3)
    s.view(B, Hkv, n, G, -1).masked_fill_(~seen[:, None, :, None, :], -math.inf)
    top = s.amax(3, keepdim=True)
    if prefix:
        # the shared keys once for all rows
        first, slot = torch.arange(prefix, device=DEV) // st["page"], torch.arange(prefix, device=DEV) % st["page"]
        kp, vp = (_fetched(st, name, st["table"][0].long()[first], slot).permute(1, 0, 2) for name in ("k", "v"))
        sp = q.transpose(0, 1).reshape(Hkv, B * n * G, D) @ kp.transpose(1, 2)
        top = torch.maximum(top, sp.amax(2).view(Hkv, B, n * G, 1).transpose(0, 1))
    # a row that sees nothing: a sum of zero, and zeros
    top = torch.where(top > -math.inf, top, torch.zeros_like(top))
    p = s.sub_(top).exp_()
    total = p.sum(3, keepdim=True)
    o = p @ vx
    if prefix:
        p = (sp.view(Hkv, B, n * G, prefix) - top.transpose(0, 1)).exp_()
        total = total + p.sum(3, keepdim=True).transpose(0, 1)
        o = o + (p.view(Hkv, B * n * G, prefix) @ vp).view(Hkv, B, n * G, D).transpose(0, 1)
    o = torch.where(total > 0, o / total, torch.zeros_like(o))
    back = lambda x: x.view(B, Hkv, n, G, -1).permute(0, 2, 1, 3, 4).reshape(B, n, Hq, -1)[seq, row]
    lse = back(top + total.log())[..., 0] if st["lse"] else None
    return _answer(back(o).to(torch.bfloat16), lse)


# ------------------------------------------------------------------ work

def work(case):
    Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
    if case["op"] == "norm_rope":
        T = case["T"]
        return {"bytes": 4 * T * (Hq + Hkv) * D + 4 * T + 4 * case["rot"], "flops": 8 * T * (Hq + Hkv) * D}
    new, kv = _lengths(case)
    T = sum(new)
    token = 2 * Hkv * (2 * D if case["fmt"] == "bf16" else D + 4)       # a cached token's key and value, scales with them
    lists = 8 * case["B"]
    if case["op"] == "append":
        pages = sum((k - 1) // case["page"] - (k - n) // case["page"] + 1 for n, k in zip(new, kv))
        by = T * (2 * (Hq + 2 * Hkv) * D + 2 * Hq * D + token) + lists + 4 * pages + 4 * case["rot"]
        return {"bytes": by, "flops": 8 * T * (Hq + Hkv) * D}
    window, sinks, prefix = case.get("window", 0), case.get("sinks", 0), case.get("prefix", 0)
    keys, pairs = prefix, prefix * T
    for n, k in zip(new, kv):
        p = k - n                                                       # the first new token's position
        if window:
            keys += k - max(0, p - window + 1) + min(sinks, max(0, p - window + 1))
            # of the position's p + 1 tokens the last `window`, and the first ones before those
            pairs += sum(min(p + i + 1, window) + min(sinks, max(0, p + i + 1 - window)) for i in range(n))
        else:
            keys += k - prefix
            pairs += n * (p - prefix) + n * (n + 1) // 2
    by = 4 * T * Hq * D + keys * token + 4 * (keys // case["page"]) + lists + (4 * T * Hq if case["lse"] else 0)
    return {"bytes": by, "flops": 4 * pairs * Hq * D}


# ------------------------------------------------------------------ the definitions in 64 bits

def exact(case, seed):
    st = prepare(case, seed)
    d = torch.float64
    Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
    G = Hq // Hkv

    def cached(name):
        if case["fmt"] == "bf16":
            return st[name].to(d)
        return st[name].view(torch.float8_e4m3fn).to(d) * st[name + "_scale"].to(d)[..., None]

    def turned(x, w, positions):
        """The norm's quotient times its weight, and each pair as a complex number times exp(i angle)."""
        x = x.to(d)
        if w is not None:
            x = w.to(d) * x / torch.sqrt(torch.linalg.vector_norm(x, dim=2, keepdim=True).square() / D + EPS)
        r = case["rot"]
        pairs = x[..., :r].reshape(*x.shape[:2], r // 2, 2) if case["inter"] else \
            torch.stack(x[..., :r].split(r // 2, dim=2), 3)
        half = torch.arange(r // 2, dtype=d, device=DEV) / (r // 2)
        angle = positions.to(d)[:, None] * torch.pow(torch.tensor(BASE, dtype=d, device=DEV), -half)
        z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * torch.polar(torch.ones_like(angle), angle)[:, None])
        z = z.flatten(2) if case["inter"] else torch.cat((z[..., 0], z[..., 1]), 2)
        return torch.cat((z, x[..., r:]), 2)

    if case["op"] == "norm_rope":
        q, k, _ = _heads(st)
        return {"q": turned(q, st["wq"], st["positions"]), "k": turned(k, st["wk"], st["positions"])}
    new, kv = _lengths(case)
    table = st["table"].cpu()
    if case["op"] == "append":
        q, k, v = _heads(st)
        positions = torch.cat([torch.arange(m - n, m) for n, m in zip(new, kv)])
        seq = torch.repeat_interleave(torch.arange(case["B"]), torch.tensor(new))
        page = table[seq, positions // case["page"]].long().to(DEV)
        slot = (positions % case["page"]).to(DEV)
        positions = positions.to(DEV)
        out = {"q": turned(q, st["wq"], positions)}
        for name, x in (("k", turned(k, st["wk"], positions)), ("v", v.to(d))):
            if case["fmt"] == "bf16":
                out[name] = st[name].to(d)
                out[name][page, :, slot] = x
            else:
                # a code stands for the quotient within half a step
                s = torch.linalg.vector_norm(x, ord=math.inf, dim=2) / 448.0
                out[name], out[name + "_scale"] = st[name].view(torch.float8_e4m3fn).to(d), st[name + "_scale"].to(d)
                out[name][page, :, slot] = x / s[..., None]
                out[name + "_scale"][page, :, slot] = s
        return out
    T, window, sinks = st["T"], case.get("window", 0), case.get("sinks", 0)
    k_all, v_all = cached("k"), cached("v")
    out = torch.zeros((T, Hq, D), dtype=d, device=DEV)
    lse = torch.zeros((T, Hq), dtype=d, device=DEV)
    at = 0
    for b, (n, m) in enumerate(zip(new, kv)):
        pages = table[b, :(m + case["page"] - 1) // case["page"]].long().to(DEV)
        q = st["q"][at:at + n].to(d)
        key, query = torch.arange(m, device=DEV)[None, :], torch.arange(m - n, m, device=DEV)[:, None]
        hidden = key > query
        if window:
            hidden = hidden | ((query - key >= window) & (key >= sinks))
        for h in range(Hkv):
            k, v = (x[pages, h].reshape(-1, D)[:m] for x in (k_all, v_all))
            heads = range(h * G, (h + 1) * G) if n * m > 1 << 20 else [slice(h * G, (h + 1) * G)]
            for j in heads:
                s = torch.tensordot(q[:, j], k, dims=([-1], [1])) / math.sqrt(D)
                s = torch.where(hidden if s.dim() == 2 else hidden[:, None, :], -math.inf, s)
                out[at:at + n, j] = torch.softmax(s, -1) @ v
                lse[at:at + n, j] = torch.logsumexp(s, -1)
        at += n
    return _answer(out, lse if case["lse"] else None)
