"""Cases of the operators that stand between the quantized products of a decoder block.

  norm      h = x + residual, y = rms_norm(h) * weight, as bf16 or as 8-bit codes with a scale per row
  swiglu    y = silu(gate) * up of the fused gate_up output, in the same forms
  dispatch  top-k expert ids -> offsets, the row of every (token, choice) slot, the tokens' rows sorted by expert
  combine   the experts' rows back to their tokens, weighted and added to the residual; and its gradient
  linear    y = act(a . w_hat + bias) + residual for INT4 g128 weights

`own` chooses between the plain torch form of each operator and the library's entry points.  Sizes are those of the
repository's workloads: hidden 4096 / 8192 and intermediate 14336 / 28672 dense layers, experts of hidden 2048 with
top-8 of 128, batches from one token to the thousands of a prefill.
"""
import math

import torch

own = False

DEV = "cuda"
EPS = 1e-5
QMAX = {"e4m3": 448.0, "int8": 127.0}


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one decode token entering a W8A8-FP8 projection
        {"name": "norm 1 x 4096 e4m3", "op": "norm", "M": 1, "K": 4096, "out": "e4m3", "residual": True},
        # a prefill chunk of a wide model, bf16 for a W4A16 projection; an odd number of rows
        {"name": "norm 8191 x 8192 bf16", "op": "norm", "M": 8191, "K": 8192, "out": "bf16", "residual": True},
        # the largest decode batch, entering a W8A8-INT8 down projection
        {"name": "swiglu 16 x 14336 int8", "op": "swiglu", "M": 16, "I": 14336, "out": "int8"},
        # a prefill chunk entering a W8A8-FP8 down projection
        {"name": "swiglu 4097 x 14336 e4m3", "op": "swiglu", "M": 4097, "I": 14336, "out": "e4m3"},
        # a few decode tokens to the experts, bf16 rows for the grouped W4A16 product
        {"name": "dispatch 4 bf16", "op": "dispatch", "B": 4, "k": 8, "E": 128, "K": 2048, "out": "bf16", "dropped": 0.0},
        # a prefill batch with padded tokens, e4m3 rows and scales for the grouped W4A8 product
        {"name": "dispatch 8192 e4m3", "op": "dispatch", "B": 8192, "k": 8, "E": 128, "K": 2048, "out": "e4m3", "dropped": 0.05},
        # one decode token back from its experts
        {"name": "combine 1", "op": "combine", "B": 1, "k": 8, "E": 128, "K": 2048, "residual": True, "dropped": 0.0},
        # a prefill batch back from its experts
        {"name": "combine 8192", "op": "combine", "B": 8192, "k": 8, "E": 128, "K": 2048, "residual": True, "dropped": 0.05},
        # the router's training over frozen experts: an odd batch with padded tokens
        {"name": "combine backward 4099", "op": "combine_backward", "B": 4099, "k": 8, "E": 128, "K": 2048, "dropped": 0.05},
        # qkv with a bias, one decode token
        {"name": "linear 1 x 4096 x 6144 bias", "op": "linear", "M": 1, "K": 4096, "N": 6144, "bias": True, "act": "none",
         "residual": False},
        # the down projection added to the residual stream, the largest decode batch
        {"name": "linear 16 x 14336 x 4096 res", "op": "linear", "M": 16, "K": 14336, "N": 4096, "bias": False, "act": "none",
         "residual": True},
        # the first product of an ungated feed-forward layer, an odd large batch
        {"name": "linear 1000 x 4096 x 14336 gelu", "op": "linear", "M": 1000, "K": 4096, "N": 14336, "bias": True,
         "act": "gelu", "residual": False},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "swiglu", "dispatch", "combine", "combine_backward", "linear"])
    if op == "norm":
        K = 8 * _log(rng, 8, 2048)
        M = _log(rng, 1, min(32768, 8191 * 8192 // K))
        return {"op": op, "M": M, "K": K, "out": rng.choice(["bf16", "e4m3", "int8"]), "residual": rng.random() < 0.7}
    if op == "swiglu":
        n = 8 * _log(rng, 16, 3584)
        M = _log(rng, 1, min(32768, 4097 * 14336 // n))
        return {"op": op, "M": M, "I": n, "out": rng.choice(["bf16", "e4m3", "int8"])}
    if op == "linear":
        K = 128 * _log(rng, 2, 112)
        N = 16 * _log(rng, 8, 896)
        M = _log(rng, 1, min(1000, 1000 * 4096 * 14336 // (K * N)))
        return {"op": op, "M": M, "K": K, "N": N, "bias": rng.random() < 0.6,
                "act": rng.choice(["none", "relu", "gelu", "gelu_tanh", "silu"]), "residual": rng.random() < 0.6}
    E = rng.choice([8, 16, 60, 64, 128, 256])
    k = rng.randint(1, 8)
    K = 8 * _log(rng, 16, 1024)
    B = _log(rng, 1, min(32768, 8192 * 8 * 2048 // (2 * k * K)))
    case = {"op": op, "B": B, "k": k, "E": E, "K": K, "dropped": rng.choice([0.0, 0.0, 0.1])}
    if op == "dispatch":
        case["out"] = rng.choice(["bf16", "e4m3"])
    if op == "combine":
        case["residual"] = rng.random() < 0.5
    return case


# ------------------------------------------------------------------ inputs

def _hidden(g, M, K):
    """A residual stream: normal values, a few channels larger than the others."""
    gain = torch.exp(0.5 * torch.randn(K, generator=g, device=DEV))
    return (torch.randn((M, K), generator=g, device=DEV) * gain).to(torch.bfloat16)


def _routing(g, case):
    """Top-k expert ids of a router that likes some experts more, softmax weights over the chosen; dropped slots are -1."""
    B, k, E = case["B"], case["k"], case["E"]
    logits = torch.randn((B, E), generator=g, device=DEV) + 0.5 * torch.randn(E, generator=g, device=DEV)
    top, ids = torch.topk(logits, k, dim=1)
    drop = torch.rand((B, k), generator=g, device=DEV) < case["dropped"]
    ids = torch.where(drop, torch.full_like(ids, -1), ids).to(torch.int32).contiguous()
    return ids, torch.softmax(top, dim=1).contiguous()


def _rows_by_expert(ids, E):
    """offsets [E + 1] and the row of every slot (-1: no row): slots in order inside an expert, experts ascending."""
    flat = ids.reshape(-1).long()
    kept = (flat >= 0) & (flat < E)
    key = torch.where(kept, flat, torch.full_like(flat, E))
    _, order = torch.sort(key, stable=True)
    row = torch.empty_like(flat)
    row[order] = torch.arange(flat.numel(), device=flat.device)
    row = torch.where(kept, row, torch.full_like(row, -1)).to(torch.int32)
    offsets = (key[None, :] < torch.arange(E + 1, device=flat.device)[:, None]).sum(1).to(torch.int32)
    return offsets, row.reshape(ids.shape)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    op = case["op"]
    st = dict(case)
    bf16 = dict(dtype=torch.bfloat16, device=DEV)
    if op == "norm":
        M, K = case["M"], case["K"]
        st["x"] = _hidden(g, M, K)
        st["r"] = _hidden(g, M, K) if case["residual"] else None
        st["w"] = (1 + 0.1 * torch.randn(K, generator=g, device=DEV)).to(torch.bfloat16)
        st["h"] = torch.empty((M, K), **bf16) if case["residual"] else None
        _outputs(st, M, K)
    elif op == "swiglu":
        M, n = case["M"], case["I"]
        st["gu"] = (1.5 * torch.randn((M, 2 * n), generator=g, device=DEV)).to(torch.bfloat16)
        _outputs(st, M, n)
    elif op == "linear":
        M, K, N = case["M"], case["K"], case["N"]
        st["a"] = torch.randn((M, K), generator=g, device=DEV).to(torch.bfloat16)
        # codes of normal weights whose group maximum is near 3 standard deviations, eight to a word
        words = torch.zeros(K * N // 8, dtype=torch.int32, device=DEV)
        for p in range(8):
            code = (torch.randn(K * N // 8, generator=g, device=DEV) * (7 / 3)).round_().clamp_(-7, 7).to(torch.int32) + 8
            words |= code << (4 * p)
        st["packed"] = words
        st["scales"] = (0.02 * 3 / 7 * (0.8 + 0.4 * torch.rand(K // 128 * N, generator=g, device=DEV))).to(torch.bfloat16)
        st["b"] = (0.5 * torch.randn(N, generator=g, device=DEV)).to(torch.bfloat16) if case["bias"] else None
        st["r"] = torch.randn((M, N), generator=g, device=DEV).to(torch.bfloat16) if case["residual"] else None
        st["y"] = torch.empty((M, N), **bf16)
        if own:
            from weight_only_quantized_w4a16_amd import ops
            st["ws_bytes"] = ops.w4a16_workspace_bytes(M, N, K)
            st["ws"] = torch.zeros(st["ws_bytes"], dtype=torch.uint8, device=DEV) if st["ws_bytes"] else None
    else:
        B, k, E, K = case["B"], case["k"], case["E"], case["K"]
        ids, weights = _routing(g, case)
        if op == "dispatch":
            st["ids"] = ids
            st["offsets"] = torch.empty(E + 1, dtype=torch.int32, device=DEV)
            st["row"] = torch.empty((B, k), dtype=torch.int32, device=DEV)
            x = _hidden(g, B, K)
            if case["out"] == "e4m3":
                s = x.float().abs().amax(1).clamp_min(1e-12) / 448.0
                st["x"] = (x.float() / s[:, None]).clamp_(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
                st["s"] = s
                st["rows"] = torch.zeros((B * k, K), dtype=torch.uint8, device=DEV)
                st["rs"] = torch.zeros(B * k, dtype=torch.float32, device=DEV)
            else:
                st["x"], st["s"], st["rs"] = x, None, None
                st["rows"] = torch.zeros((B * k, K), **bf16)
            if own:
                from weight_only_quantized_w4a16_amd import ops
                st["ws_bytes"] = ops.moe_dispatch_workspace_bytes(B, k, E)
                st["ws"] = torch.empty(st["ws_bytes"], dtype=torch.uint8, device=DEV) if st["ws_bytes"] else None
        else:
            st["row"] = _rows_by_expert(ids, E)[1]
            st["weights"] = weights
            st["rows"] = torch.randn((B * k, K), generator=g, device=DEV).to(torch.bfloat16)
            if op == "combine":
                st["r"] = _hidden(g, B, K) if case["residual"] else None
                st["y"] = torch.empty((B, K), **bf16)
            else:
                st["dy"] = (0.01 * torch.randn((B, K), generator=g, device=DEV)).to(torch.bfloat16)
                st["drows"] = torch.zeros((B * k, K), **bf16)
                st["dw"] = torch.empty((B, k), dtype=torch.float32, device=DEV)
    return st


def _outputs(st, M, K):
    if st["out"] == "bf16":
        st["y"] = torch.empty((M, K), dtype=torch.bfloat16, device=DEV)
    else:
        st["q"] = torch.empty((M, K), dtype=torch.uint8 if st["out"] == "e4m3" else torch.int8, device=DEV)
        st["s"] = torch.empty(M, dtype=torch.float32, device=DEV)
        if st["out"] == "int8":
            st["v"] = torch.empty((M, K), dtype=torch.bfloat16, device=DEV)


# ------------------------------------------------------------------ one pass

def run(state):
    return (_run_own if own else _run_plain)(state)


def _codes(st):
    """Codes as the values they stand for: e4m3 codes as e4m3 numbers beside their scales, int8 ones times their scales."""
    if st["out"] == "e4m3":
        return {"q": st["q"].view(torch.float8_e4m3fn), "s": st["s"]}
    torch.mul(st["q"], st["s"][:, None], out=st["v"])
    return {"v": st["v"]}


def _run_own(st):
    from weight_only_quantized_w4a16_amd import ops
    op = st["op"]
    if op == "norm":
        M, K = st["M"], st["K"]
        if st["out"] == "bf16":
            ops.rms_norm(st["x"], st["r"], st["w"], EPS, M, K, st["h"], st["y"])
            out = {"y": st["y"]}
        else:
            f = ops.rms_norm_quant if st["out"] == "e4m3" else ops.rms_norm_quant_int8
            f(st["x"], st["r"], st["w"], EPS, M, K, st["h"], None, st["q"], st["s"])
            out = _codes(st)
        if st["h"] is not None:
            out["h"] = st["h"]
        return out
    if op == "swiglu":
        if st["out"] == "bf16":
            ops.swiglu(st["gu"], st["M"], st["I"], st["y"])
            return {"y": st["y"]}
        f = ops.swiglu_quant if st["out"] == "e4m3" else ops.swiglu_quant_int8
        f(st["gu"], st["M"], st["I"], st["q"], st["s"])
        return _codes(st)
    if op == "linear":
        ops.qgemm_w4a16_epilogue(st["a"], st["packed"], st["scales"], st["b"], st["act"], st["r"], st["y"], st["M"], st["N"],
                                 st["K"], st["ws"], st["ws_bytes"])
        return {"y": st["y"]}
    B, k, E, K = st["B"], st["k"], st["E"], st["K"]
    if op == "dispatch":
        ops.moe_dispatch(st["ids"], st["x"], st["s"], B, k, E, K if st["out"] == "e4m3" else 2 * K, st["offsets"], st["row"],
                         st["rows"], st["rs"], st["ws"], st["ws_bytes"])
        return _dispatched(st, st["offsets"], st["row"], st["rows"], st["rs"])
    if op == "combine":
        ops.moe_combine(st["rows"], st["row"], st["weights"], st["r"], B, k, K, st["y"])
        return {"y": st["y"]}
    ops.moe_combine_backward(st["dy"], st["rows"], st["row"], st["weights"], B, k, K, st["drows"], st["dw"])
    return {"drows": st["drows"], "dw": st["dw"]}


def _dispatched(st, offsets, row, rows, rs):
    if st["out"] == "e4m3":
        return {"offsets": offsets, "row": row, "rows": rows.view(torch.float8_e4m3fn), "rs": rs}
    return {"offsets": offsets, "row": row, "rows": rows}


def _plain_codes(st, y):
    s = y.abs().amax(1) / QMAX[st["out"]]
    q = y / torch.where(s > 0, s, torch.ones_like(s))[:, None]
    if st["out"] == "e4m3":
        return {"q": q.clamp(-448, 448).to(torch.float8_e4m3fn), "s": s}
    return {"v": (q.round().clamp(-127, 127) * s[:, None]).to(torch.bfloat16)}


def _act(x, act):
    if act == "relu":
        return torch.clamp_min(x, 0)
    if act == "gelu":
        return 0.5 * x * (1 + torch.erf(x * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * x * (1 + torch.tanh(math.sqrt(2 / math.pi) * (x + 0.044715 * x * x * x)))
    if act == "silu":
        return x / (1 + torch.exp(-x))
    return x


# bits of row i's code inside a word: slots 0..3 hold rows 0, 2, 4, 6, slots 4..7 rows 1, 3, 5, 7
SHIFTS = (0, 16, 4, 20, 8, 24, 12, 28)


def _run_plain(st):
    op = st["op"]
    bf16 = torch.bfloat16
    if op == "norm":
        h = st["x"].float()
        if st["r"] is not None:
            h = h + st["r"].float()
        y = h * torch.rsqrt((h * h).mean(1, keepdim=True) + EPS) * st["w"].float()
        out = {"y": y.to(bf16)} if st["out"] == "bf16" else _plain_codes(st, y)
        if st["r"] is not None:
            out["h"] = h.to(bf16)
        return out
    if op == "swiglu":
        gu = st["gu"].float()
        gate, up = gu[:, :st["I"]], gu[:, st["I"]:]
        y = gate / (1 + torch.exp(-gate)) * up
        return {"y": y.to(bf16)} if st["out"] == "bf16" else _plain_codes(st, y)
    if op == "linear":
        K, N = st["K"], st["N"]
        G, NT = K // 128, N // 16
        # native order: [column tile, group, k quarter, column, k step] words of 8 rows
        words = st["packed"].view(NT, G, 4, 16, 4)
        shifts = torch.tensor(SHIFTS, dtype=torch.int32, device=words.device)
        w = ((words[..., None] >> shifts) & 15).to(torch.float32) - 8
        w = w * st["scales"].view(NT, G, 1, 16, 1, 1).float()
        w = w.permute(1, 4, 2, 5, 0, 3).reshape(K, N)
        y = st["a"].float() @ w
        if st["b"] is not None:
            y = y + st["b"].float()
        y = _act(y, st["act"])
        if st["r"] is not None:
            y = y + st["r"].float()
        return {"y": y.to(bf16)}
    B, k, E, K = st["B"], st["k"], st["E"], st["K"]
    if op == "dispatch":
        offsets, row = _rows_by_expert(st["ids"], E)
        flat = row.reshape(-1).long()
        # slots without a row write one spare row past the end
        at = torch.where(flat >= 0, flat, torch.full_like(flat, B * k))
        rows = torch.zeros((B * k + 1, K), dtype=st["rows"].dtype, device=flat.device)
        rows[at] = st["x"].repeat_interleave(k, 0)
        rs = None
        if st["s"] is not None:
            rs = torch.zeros(B * k + 1, dtype=torch.float32, device=flat.device)
            rs[at] = st["s"].repeat_interleave(k, 0)
            rs = rs[:-1]
        return _dispatched(st, offsets, row, rows[:-1], rs)
    kept = st["row"] >= 0
    at = st["row"].clamp_min(0).long()
    w = torch.where(kept, st["weights"], torch.zeros_like(st["weights"]))
    if op == "combine":
        y = (st["rows"][at].float() * w[:, :, None]).sum(1)
        if st["r"] is not None:
            y = y + st["r"].float()
        return {"y": y.to(bf16)}
    dy = st["dy"].float()
    dw = (st["rows"][at].float() * dy[:, None, :]).sum(2)
    dw = torch.where(kept, dw, torch.zeros_like(dw))
    spare = torch.where(kept, st["row"].long(), torch.full_like(at, B * k))
    drows = torch.zeros((B * k + 1, K), dtype=bf16, device=dy.device)
    drows[spare.reshape(-1)] = (w[:, :, None] * dy[:, None, :]).to(bf16).reshape(B * k, K)
    return {"drows": drows[:-1], "dw": dw}


# ------------------------------------------------------------------ work

def work(case):
    op = case["op"]
    width = {"bf16": 2, "e4m3": 1, "int8": 1}
    if op == "norm":
        n = case["M"] * case["K"]
        by = n * (2 + (4 if case["residual"] else 0) + width[case["out"]]) + 2 * case["K"]
        by += 4 * case["M"] if case["out"] != "bf16" else 0
        return {"bytes": by, "flops": 6 * n}
    if op == "swiglu":
        n = case["M"] * case["I"]
        return {"bytes": n * (4 + width[case["out"]]) + (4 * case["M"] if case["out"] != "bf16" else 0), "flops": 6 * n}
    if op == "linear":
        M, K, N = case["M"], case["K"], case["N"]
        by = K * N // 2 + 2 * (K // 128) * N + 2 * M * K + 2 * M * N
        by += (2 * N if case["bias"] else 0) + (2 * M * N if case["residual"] else 0)
        return {"bytes": by, "flops": 2 * M * N * K}
    B, k, K = case["B"], case["k"], case["K"]
    T = max(1, round(B * k * (1 - case["dropped"])))
    if op == "dispatch":
        row = K * width[case["out"]] + (4 if case["out"] == "e4m3" else 0)
        return {"bytes": 8 * B * k + 4 * case["E"] + (B + T) * row, "flops": 0}
    if op == "combine":
        return {"bytes": 8 * B * k + 2 * K * (T + B * (2 if case["residual"] else 1)), "flops": 2 * T * K}
    return {"bytes": 12 * B * k + 2 * K * (B + 2 * T), "flops": 3 * T * K}


# ------------------------------------------------------------------ the definitions in 64 bits

def exact(case, seed):
    st = prepare(case, seed)
    op = st["op"]
    d = torch.float64
    if op in ("norm", "swiglu"):
        if op == "norm":
            h = st["x"].to(d) if st["r"] is None else st["x"].to(d).add_(st["r"].to(d))
            norm = torch.linalg.vector_norm(h, dim=1).square() / case["K"]
            y = st["w"].to(d) * (h / torch.sqrt(norm + EPS)[:, None])
        else:
            gate, up = st["gu"].to(d).split(case["I"], dim=1)
            y, h = gate * torch.sigmoid(gate) * up, None
        if case["out"] == "bf16":
            out = {"y": y}
        else:
            top = torch.maximum(y.amax(1), -y.amin(1))
            s = top / QMAX[case["out"]]
            # an e4m3 code stands for the quotient within half a step, an int8 code for a whole number of scales
            quotient = y / s[:, None]
            out = {"q": quotient, "s": s} if case["out"] == "e4m3" else {"v": torch.round(quotient) * s[:, None]}
        if op == "norm" and st["r"] is not None:
            out["h"] = h
        return out
    if op == "linear":
        M, K, N = case["M"], case["K"], case["N"]
        G = K // 128
        words = st["packed"].to(torch.int64) & 0xFFFFFFFF
        k = torch.arange(K, device=DEV)[:, None]
        y = torch.empty((M, N), dtype=d, device=DEV)
        for n0 in range(0, N, 2048):
            n = torch.arange(n0, min(N, n0 + 2048), device=DEV)[None, :]
            tile = (n // 16) * G + k // 128
            i = k % 8
            slot = torch.where(i % 2 == 0, i // 2, 4 + i // 2)
            word = words[tile * 256 + ((k % 32) // 8 * 16 + n % 16) * 4 + (k % 128) // 32]
            code = torch.div(word, 16 ** slot, rounding_mode="floor") % 16
            w = (code - 8).to(d) * st["scales"].to(d)[tile * 16 + n % 16]
            y[:, n0:n0 + w.shape[1]] = st["a"].to(d) @ w
        if st["b"] is not None:
            y += st["b"].to(d)
        if case["act"] == "relu":
            y = torch.where(y > 0, y, torch.zeros_like(y))
        elif case["act"] == "gelu":
            y = y * torch.special.ndtr(y)
        elif case["act"] == "gelu_tanh":
            y = y * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (y + 0.044715 * y ** 3))
        elif case["act"] == "silu":
            y = y * torch.sigmoid(y)
        if st["r"] is not None:
            y += st["r"].to(d)
        return {"y": y}
    B, k, E, K = case["B"], case["k"], case["E"], case["K"]
    if op == "dispatch":
        # counting, expert by expert, on the host
        flat = st["ids"].reshape(-1).cpu()
        rows = torch.zeros((B * k, K), dtype=d, device=DEV)
        rs = torch.zeros(B * k, dtype=d, device=DEV)
        row, at = torch.full((B * k,), -1, dtype=torch.int32), 0
        offsets = torch.zeros(E + 1, dtype=torch.int32)
        x = st["x"].view(torch.float8_e4m3fn).to(d) if case["out"] == "e4m3" else st["x"].to(d)
        for e in range(E):
            mine = torch.nonzero(flat == e).reshape(-1)
            row[mine] = torch.arange(at, at + mine.numel(), dtype=torch.int32)
            rows[at:at + mine.numel()] = x[(mine // k).to(DEV)]
            if case["out"] == "e4m3":
                rs[at:at + mine.numel()] = st["s"].to(d)[(mine // k).to(DEV)]
            at += mine.numel()
            offsets[e + 1] = at
        out = {"offsets": offsets.to(DEV), "row": row.reshape(B, k).to(DEV), "rows": rows}
        if case["out"] == "e4m3":
            out["rs"] = rs
        return out
    y = torch.zeros((B, K), dtype=d, device=DEV) if op == "combine" else None
    drows = torch.zeros((B * k, K), dtype=d, device=DEV)
    dw = torch.zeros((B, k), dtype=d, device=DEV)
    for j in range(k):
        b = torch.nonzero(st["row"][:, j] >= 0).reshape(-1)
        r = st["row"][b, j].long()
        w = st["weights"][b, j].to(d)
        if op == "combine":
            y[b] += w[:, None] * st["rows"][r].to(d)
        else:
            drows[r] = w[:, None] * st["dy"][b].to(d)
            dw[b, j] = torch.linalg.vecdot(st["dy"][b].to(d), st["rows"][r].to(d))
    if op == "combine":
        return {"y": y if st["r"] is None else y + st["r"].to(d)}
    return {"drows": drows, "dw": dw}
