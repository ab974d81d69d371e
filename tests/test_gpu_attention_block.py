"""The attention half of a decoder block as it is used: qkv product, append, attention, o product; prefill and then decode
steps, captured graphs, streams, one workspace for many shapes, long caches, and lists that name nothing valid."""
import numpy as np
import pytest
import torch

from attention_helpers import Batch, attend, bf16, check
from gpu_helpers import announce
from oracle import attention as oracle
from oracle import fp8_e4m3 as f8

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ops():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    from weight_only_quantized_w4a16_amd import ops as _ops
    return _ops


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def values(cache):
    """The cache as float64 (keys, values)."""
    if cache.fmt == "bf16":
        return cache.k.double().cpu().numpy(), cache.v.double().cpu().numpy()
    return tuple(f8.e4m3_decode(c.cpu().numpy()).astype(np.float64) * s.double().cpu().numpy()[..., None]
                 for c, s in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)))


def make(ops, fmt, window=0, sinks=0, Hq=4, Hkv=2, D=64, pages=40, page=16, seed=0):
    rng = np.random.default_rng(seed)
    cache = ops.PagedKVCache(pages, Hkv, D, page, fmt)
    for t in (cache.k, cache.v):
        t.view(torch.uint8).fill_(0x7f)                      # NaN in e4m3, a large number in bf16
    w = [bf16(1 + 0.3 * rng.standard_normal(D))[1].cuda() for _ in range(2)]
    layer = ops.PagedAttention(cache, Hq, ops.rotary_frequencies(D, 10000.0), *w, window=window, sinks=sinks)
    return cache, layer, rng


def close(out, want, what):
    """The outputs of attend (flattened heads) against the oracle's, where the cache is what the GPU holds: the rounding of
    the probabilities and of the output, 2^-8 each, and fp32 work (sums of at most 300 products of magnitudes below 2^7)."""
    y, _, mean, _ = want
    got = out.double().cpu().numpy().reshape(y.shape)
    live = ~np.isnan(mean).any(-1)
    bound = (2.0 ** -8 + 2.0 ** -12) * mean + 2.0 ** -8 * (1 + 2.0 ** -6) * np.abs(y) + 1e-6
    assert (np.abs(got - y) <= bound)[live].all(), what


@pytest.mark.parametrize("fmt,window,sinks", [("bf16", 0, 0), ("e4m3", 0, 0), ("bf16", 24, 3)])
def test_prefill_then_decode_between_products(ops, fmt, window, sinks):
    cache, layer, rng = make(ops, fmt, window, sinks)
    K, width = 128, (4 + 4) * 64
    qkv_w = ops.Int4G128Weight.from_bf16(bf16(rng.standard_normal((K, width)) * 0.1)[1].cuda())
    o_w = ops.Int4G128Weight.from_bf16(bf16(rng.standard_normal((256, K)) * 0.1)[1].cuda())
    qkv_proj, o_proj = ops.W4A16Linear(qkv_w), ops.W4A16Linear(o_w)
    table = torch.from_numpy(rng.permutation(40)[:36].reshape(3, 12).astype(np.int32)).cuda()
    length = np.zeros(3, np.int64)
    for new in ([30, 1, 55], [1, 1, 1], [1, 0, 1], [3, 2, 1], [1, 1, 1]):
        length += new
        T = sum(new)
        offsets, kv = i32(np.concatenate([[0], np.cumsum(new)]).tolist()), i32(length.tolist())
        x = bf16(rng.standard_normal((T, K)))[1].cuda()
        qkv = qkv_proj(x)
        announce(f"block {fmt} window {window} new={new}")
        q = layer.append(qkv, table, offsets, kv)
        y = layer.attend(q, table, offsets, kv, max(new))
        out = o_proj(y, residual=x)
        assert torch.isfinite(out).all()
        k, v = values(cache)
        want = oracle.paged_attention(q.double().cpu().numpy(), k, v, table.cpu().numpy(), offsets.cpu().numpy(),
                                      kv.cpu().numpy(), 0.125, window, sinks)
        close(y, want, f"{fmt} {new}")
        # the whole call in one, on the same cache rows: the same bits
        again = layer(qkv, table, offsets, kv, max(new))
        assert torch.equal(again, y)
        # keys of the new tokens, from the product's own output
        heads = qkv.double().cpu().numpy().reshape(T, 8, 64)
        seq, pos = oracle.places(T, offsets.cpu().numpy(), kv.cpu().numpy())
        key = oracle.norm_rope(heads[:, 4:6], layer.k_weight.double().cpu().numpy(), 1e-6, pos,
                               10000.0 ** (-np.arange(32) / 32), 64, False)
        tb = table.cpu().numpy()
        got = np.stack([k[tb[s, p // 16], :, p % 16] for s, p in zip(seq, pos)])
        step = 2.0 ** -8 if fmt == "bf16" else 2.0 ** -4
        top = np.abs(key).max(-1, keepdims=True)
        assert (np.abs(got - key) <= step * 1.02 * np.abs(key) + 2.0 ** -18 * top).all()


def test_decode_step_in_a_captured_graph(ops):
    """Append and attention of a decode step, replayed over a growing cache with the program's own work between the
    replays; every replay equals the eager calls."""
    for fmt, shared in (("bf16", 0), ("e4m3", 0), ("bf16", 640)):
        cache, layer, rng = make(ops, fmt, pages=400, seed=3)
        _, eager, _ = make(ops, fmt, pages=400, seed=3)
        B, width = 4, 64
        table = torch.from_numpy(rng.permutation(400)[:B * width].reshape(B, width).astype(np.int32)).cuda()
        table[:, :shared // 16] = table[0, :shared // 16]
        kv = i32([900, 700, 1000, 650])
        offsets = i32([0, 1, 2, 3, 4])
        # the sequences' positions so far
        full = bf16(rng.standard_normal((B * 1000, 8 * 64)))[1].cuda()
        fill = i32([1000 * b for b in range(B + 1)])
        layer.append(full, table, fill, i32([1000] * B))
        qkv = bf16(rng.standard_normal((B, 8 * 64)))[1].cuda()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            layer(qkv, table, offsets, kv, 1, shared)
        torch.cuda.current_stream().wait_stream(side)
        eager.cache.k.copy_(cache.k), eager.cache.v.copy_(cache.v)
        if fmt == "e4m3":
            eager.cache.k_scale.copy_(cache.k_scale), eager.cache.v_scale.copy_(cache.v_scale)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            y = layer(qkv, table, offsets, kv, 1, shared)
        for step in range(5):
            announce(f"replay {step} {fmt} shared={shared}")
            qkv.copy_(bf16(rng.standard_normal((B, 8 * 64)))[1])
            kv.add_(1)
            graph.replay()
            torch.cuda.synchronize()
            got = y.clone()
            want = eager(qkv, table, offsets, kv, 1, shared)
            torch.cuda.synchronize()
            assert torch.equal(got, want), step
            assert torch.equal(cache.k, eager.cache.k) and torch.equal(cache.v, eager.cache.v)


def test_two_streams(ops):
    """Two layers at once, each on its own stream with its own workspace: the bits of one after the other."""
    layers = [make(ops, f, pages=300, seed=s) for s, f in enumerate(("bf16", "e4m3"))]
    table = torch.from_numpy(np.random.default_rng(0).permutation(300)[:280].reshape(4, 70).astype(np.int32)).cuda()
    offsets, kv = i32([0, 1, 2, 3, 4]), i32([1100, 3, 777, 1024])
    rng = np.random.default_rng(1)
    fills = [bf16(rng.standard_normal((4 * 1100, 512)))[1].cuda() for _ in layers]
    for (c, layer, _), x in zip(layers, fills):
        layer.append(x, table, i32([1100 * b for b in range(5)]), i32([1100] * 4))
    qkv = [bf16(rng.standard_normal((4, 512)))[1].cuda() for _ in layers]
    alone = [layer(x, table, offsets, kv, 1) for (_, layer, _), x in zip(layers, qkv)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in layers]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for turn in range(20):
        outs = [layer(x, table, offsets, kv, 1, stream=s) for (_, layer, _), x, s in zip(layers, qkv, streams)]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, alone)), turn


def test_one_workspace_for_all_shapes(ops):
    """A workspace of the largest call serves calls of any shape in any order; the same bits as with one of their own."""
    cases = []
    for new, kv, Hq, Hkv, D, fmt, shared in (([1], [3000], 8, 1, 64, "bf16", 0), ([1] * 5, [700, 1, 900, 30, 2], 4, 2, 128, "e4m3", 0),
                                             ([150], [1900], 4, 4, 64, "bf16", 0), ([40, 1, 2], [800, 640, 1200], 8, 2, 64, "bf16", 0),
                                             ([2] + [1] * 9, [8300, 8200] + [8193] * 8, 4, 4, 64, "e4m3", 8192)):
        cases.append((Batch(new, kv, Hq, Hkv, D, 16, fmt, seed=len(cases), shared=shared), shared))
    sizes = [ops.paged_attention_workspace_bytes(b.T, b.B, b.width, b.Hq, b.Hkv, b.D, b.page, s, 0) for b, s in cases]
    ws = torch.zeros(max(sizes), dtype=torch.uint8, device="cuda")
    ws[65536:] = 0xff                                        # NaN everywhere but in the counters
    dev = [b.device() for b, _ in cases]
    own = [attend(ops, b, shared=s, d=d)[0] for (b, s), d in zip(cases, dev)]
    order = [0, 3, 1, 4, 2, 2, 0, 1, 4, 3]
    for i in order:
        (b, s), d = cases[i], dev[i]
        announce(f"workspace case {i}")
        out = torch.full((b.T, b.Hq, b.D), 7.0, dtype=torch.bfloat16, device="cuda")
        ops.paged_attention(d["q"], d["k"], d["v"], d["k_scale"], d["v_scale"], b.pages, b.page, d["q_offsets"], d["kv_len"],
                            d["table"], b.T, b.B, b.width, b.Hq, b.Hkv, b.D, b.D ** -0.5, 0, 0, s, 0, out, None, ws, ws.numel())
        torch.cuda.synchronize()
        assert torch.equal(out, own[i]) and not ws[:65536].any()


def test_cache_past_32_bit_offsets(ops):
    """Pages whose bytes lie past 4 GiB, and elements past 2^31: append and both attention kernels."""
    pages, page, Hkv, D, Hq = 140000, 256, 1, 128, 2
    assert pages * page * D > 2 ** 32
    cache = ops.PagedKVCache(pages, Hkv, D, page, "bf16")
    layer = ops.PagedAttention(cache, Hq)
    rng = np.random.default_rng(6)
    high = [pages - 1, pages - 3, 66000, pages - 7, 5, pages - 9]
    table = i32([high[:3], high[3:]])
    new, kv = [600, 580], [600, 580]
    x, xt = bf16(rng.standard_normal((sum(new), 4 * D)))
    offsets, lens = i32([0, 600, 1180]), i32(kv)
    announce("append past 32-bit offsets")
    q = layer.append(xt.cuda(), table, offsets, lens)
    torch.cuda.synchronize()
    for s, (n, row) in enumerate(zip(new, (high[:3], high[3:]))):
        for i, p in enumerate(row):
            m = min(page, n - 256 * i)
            lo = 600 * s + 256 * i
            assert torch.equal(cache.k[p, 0, :m].cpu(), xt[lo:lo + m, 2 * D:3 * D])
            assert torch.equal(cache.v[p, 0, :m].cpu(), xt[lo:lo + m, 3 * D:])
    small = {p: i for i, p in enumerate(high)}
    k, v = (torch.stack([c[p] for p in high]).double().cpu().numpy() for c in (cache.k, cache.v))
    tb = np.array([[small[p] for p in row] for row in (high[:3], high[3:])])
    for name, lo, cnt in (("tiles", 0, 1180), ("rows", 599, 1)):
        announce(f"attention past 32-bit offsets, {name}")
        if name == "tiles":
            out = layer.attend(q, table, offsets, lens)
            want = oracle.paged_attention(q[::97].double().cpu().numpy(), k, v, tb, np.array([0, 0, 0]), np.array(kv), D ** -0.5)
            rows = [5, 599, 600, 1179]
            for t in rows:
                s = 0 if t < 600 else 1
                p = t - 600 * s
                want = oracle.paged_attention(q[t:t + 1].double().cpu().numpy(), k, v, tb[s:s + 1], np.array([0, 1]), np.array([p + 1]), D ** -0.5)
                close(out[t:t + 1], want, f"row {t}")
        else:
            out = layer.attend(q[599:600].contiguous(), table[:1], i32([0, 1]), i32([600]), 1)
            want = oracle.paged_attention(q[599:600].double().cpu().numpy(), k, v, tb[:1], np.array([0, 1]), np.array([600]), D ** -0.5)
            close(out, want, "decode")


def test_lists_that_name_nothing_valid(ops):
    """Pages outside the cache, lengths past the table or below zero, offsets out of range or out of order: nothing is read or
    written out of bounds, valid sequences keep their results, and the counters are left at zero."""
    b = Batch([1, 2, 1, 20], [40, 300, 65, 90], 4, 2, 64, 16, seed=5, extra_tokens=3)
    for spots, what in (([(0, 0, -1), (1, 3, -7), (1, 9, 10 ** 6), (3, 2, b.pages), (3, 5, 2 ** 31 - 1)], "pages"),):
        for s, i, p in spots:
            b.table[s, i] = p
        want = oracle.paged_attention(b.q, b.k, b.v, b.table, b.q_offsets, b.kv_len, 0.125)
        for m in (0, 20, 1):
            announce(f"{what} max_q={m}")
            out, lse = attend(ops, b, max_q=m)
            check(b, out, lse, want, what)
        windowed = oracle.paged_attention(b.q, b.k, b.v, b.table, b.q_offsets, b.kv_len, 0.125, 30, 4)
        out, lse = attend(ops, b, window=30, sinks=4)
        check(b, out, lse, windowed, what)
    good = Batch([1, 2, 1, 20], [40, 300, 65, 90], 4, 2, 64, 16, seed=5, extra_tokens=3, junk=0.25)
    for kv in ([-5, 300, 65, 90], [40, 10 ** 6, 65, 90], [40, 2 ** 31 - 1, 65, -2 ** 31], [0, 0, 0, 0]):
        good.kv_len = np.array(kv, np.int64).astype(np.int32)
        for window in (0, 30):
            want = oracle.paged_attention(good.q, good.k, good.v, good.table, good.q_offsets, good.kv_len, 0.125, window, 4)
            for m in (0, 20):
                announce(f"lengths {kv} max_q={m} window={window}")
                out, lse = attend(ops, good, max_q=m, window=window, sinks=4)
                check(good, out, lse, want, str(kv))
    good = Batch([1, 2, 1, 20], [40, 300, 65, 90], 4, 2, 64, 16, seed=5, extra_tokens=3)
    for offsets in ([-4, 1, 3, 4, 24], [0, 1, 3, 4, 10 ** 6], [24, 3, 2, 1, 0], [0, 27, 0, 27, 0], [5, 5, 5, 5, 5], [-2 ** 31, 2 ** 31 - 1, 0, 9, 27]):
        good.q_offsets = np.array(offsets, np.int64).astype(np.int32)
        for m in (0, 20):
            announce(f"offsets {offsets} max_q={m}")
            attend(ops, good, max_q=m)                       # asserts the counters
            attend(ops, good, max_q=m, shared=32)
        d = good.device()
        x = bf16(np.ones((good.T, 8 * 64)))[1].cuda()
        q = torch.empty((good.T, 4, 64), dtype=torch.bfloat16, device="cuda")
        ops.kv_append(x, None, None, 1e-6, None, 0, False, d["q_offsets"], d["kv_len"], d["table"], good.T, good.B, good.width, 4, 2,
                      64, d["k"], d["v"], None, None, good.pages, good.page, q)
        torch.cuda.synchronize()


def test_the_same_bits_on_every_run(ops):
    for new, kv, D, fmt, shared in (([1] * 3, [3000, 900, 1400], 128, "bf16", 0), ([60, 1], [1500, 700], 64, "e4m3", 0),
                                    ([1] * 10, [8200 + 30 * i for i in range(10)], 64, "bf16", 8192)):
        b = Batch(new, kv, 8, 4, D, 16, fmt, seed=1, shared=shared)
        d = b.device()
        first = attend(ops, b, shared=shared, d=d)
        for _ in range(4):
            again = attend(ops, b, shared=shared, d=d)
            assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def test_helper_streams_and_refusals(ops):
    cache, layer, rng = make(ops, "bf16")
    offsets, kv, table = i32([0, 2]), i32([2]), i32([[3]])
    qkv = bf16(rng.standard_normal((2, 512)))[1].cuda()
    want = layer(qkv, table, offsets, kv)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = layer(qkv, table, offsets, kv, stream=s)
    s.synchronize()
    assert torch.equal(got, want)
    out, lse = layer.attend(layer.append(qkv, table, offsets, kv), table, offsets, kv, with_lse=True)
    assert torch.equal(out, want) and lse.shape == (2, 4)
    q, k = ops.norm_rope(qkv, i32([0, 1]), 4, 2, 64, layer.inv_freq, layer.q_weight, layer.k_weight)
    assert torch.equal(q, layer.append(qkv, table, offsets, kv)) and torch.equal(k[:, :], cache.k[3, :, :2].transpose(0, 1))
    with pytest.raises(ops.QGemmError):
        layer.attend(q, table, offsets, kv, shared_prefix=8)
    with pytest.raises(ValueError, match="contiguous"):
        layer.attend(q.transpose(0, 1).contiguous().transpose(0, 1), table, offsets, kv)
