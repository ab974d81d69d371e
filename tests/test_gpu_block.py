"""The operators between two products run together with them, as a decoder block
does: a dense W4A16 / W8A8-FP8 block and a mixture-of-experts block, each stage
checked against the fp64 oracle on the inputs it received; the same block captured
in a HIP graph and replayed on changing inputs; two streams at once.
"""
import numpy as np
import pytest
import torch

from gpu_helpers import REL_TOL, announce, assert_close_rms, dev_bf16, host_bits16
from oracle import block
from oracle import fp8_e4m3 as f8
from oracle import int4_g128 as q4
from oracle.bf16 import bf16_bits_to_f32
from test_gpu_norm import assert_bf16, assert_codes
from weight_only_quantized_w4a16_amd import synth

pytestmark = pytest.mark.gpu

EPS = 1e-5
HID, INTER, E, TOPK = 256, 128, 8, 3


@pytest.fixture(scope="module")
def ops():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    from weight_only_quantized_w4a16_amd import ops as _ops
    return _ops


def f64(bits):
    return bf16_bits_to_f32(bits).astype(np.float64)


def host(t):
    return f64(host_bits16(t))


def dequant(bits):
    codes, s = q4.quantize(bits)
    return q4.dequant_f32(codes, s).astype(np.float64)


def gate_floor(gu):
    """swiglu's absolute error, as test_gpu_norm derives it."""
    n = gu.shape[1] // 2
    gate = gu[:, :n]
    return 2.0 ** -148 + np.maximum(-gate, 0) * 2.0 ** -23 * np.abs(block.swiglu(gu)) + \
        np.where(gate < -87, 2.0 ** -126 * np.abs(gate * gu[:, n:]), 0.0)


@pytest.mark.parametrize("M", [1, 5, 16, 33, 130])
def test_dense_block(ops, M):
    """norm -> qkv with a bias -> o with the residual -> norm to e4m3 -> W8A8 gate_up
    -> swiglu to e4m3 -> W8A8 down."""
    announce(f"dense block M={M}")
    w_qkv, w_o = synth.weights(HID, 3 * HID, 1), synth.weights(HID, HID, 2)
    w_gu, w_d = synth.weights(HID, 2 * INTER, 3), synth.weights(INTER, HID, 4)
    bias = synth.normal_bf16((3 * HID,), 5)
    g1, g2 = synth.normal_bf16((HID,), 6), synth.normal_bf16((HID,), 7)
    x = synth.activations(M, HID, 8)
    qkv = ops.W4A16Linear(ops.Int4G128Weight.from_bf16(dev_bf16(w_qkv)), dev_bf16(bias))
    o = ops.W4A16Linear(ops.Int4G128Weight.from_bf16(dev_bf16(w_o)))
    gu, down = (ops.W8A8Fp8Linear(ops.Fp8Weight.from_bf16(dev_bf16(w))) for w in (w_gu, w_d))
    d_x = dev_bf16(x)
    y1, _ = ops.RMSNorm(dev_bf16(g1), EPS)(d_x)
    v = qkv(y1)
    att = v[:, 2 * HID:].contiguous()
    h = o(att, residual=d_x)
    q2, s2, h2 = ops.RMSNorm(dev_bf16(g2), EPS).quantized(att, residual=h)
    u = gu(att, qa=q2, sa=s2)
    q3, s3 = ops.gated_silu_quantized(u)
    y = down(torch.empty((M, INTER), dtype=torch.bfloat16, device="cuda:0"), qa=q3, sa=s3)
    torch.cuda.synchronize()
    assert_bf16(y1, block.rms_norm(f64(x), None, f64(g1), EPS)[1], "norm")
    assert_close_rms(host_bits16(v), host(y1) @ dequant(w_qkv) + f64(bias), what="qkv")
    assert_close_rms(host_bits16(h), host(att) @ dequant(w_o) + f64(x), what="o")
    assert_codes(q2, s2, block.rms_norm(host(att), host(h), f64(g2), EPS)[1], "e4m3", "norm to e4m3")
    dec = lambda q, s: f8.e4m3_decode(q.cpu().numpy()).astype(np.float64) * s.cpu().numpy().astype(np.float64)[:, None]
    qw, sw = f8.quant_weight_per_channel(w_gu)
    assert_close_rms(host_bits16(u), f8.gemm_ref(q2.cpu().numpy(), s2.cpu().numpy(), qw, sw), what="gate_up")
    assert_codes(q3, s3, block.swiglu(host(u)), "e4m3", "swiglu", gate_floor(host(u)))
    qw, sw = f8.quant_weight_per_channel(w_d)
    assert_close_rms(host_bits16(y), dec(q3, s3) @ (f8.e4m3_decode(qw).astype(np.float64) * sw), what="down")


def moe_weights(ops):
    wg = [synth.weights(HID, 2 * INTER, 20 + e) for e in range(E)]
    wd = [synth.weights(INTER, HID, 40 + e) for e in range(E)]
    stack = lambda ws: ops.GroupedInt4Weight.from_bf16(torch.stack([dev_bf16(w) for w in ws]))
    return wg, wd, stack(wg), stack(wd)


def moe_block(ops, norm, gate_up, down, x, residual, ids, weights):
    """One mixture-of-experts block in W4A8; every intermediate."""
    q, s, h, y = norm.quantized(x, residual=residual, with_bf16=True)
    routing, rq, rs = ops.MoeRouting.dispatch(ids, E, q, s)
    u = gate_up.w4a8(rq, rs, routing.offsets)
    q2, s2 = ops.gated_silu_quantized(u)
    d = down.w4a8(q2, s2, routing.offsets)
    out = routing.combine(d, weights, residual=h)
    return dict(q=q, s=s, h=h, y=y, off=routing.offsets, row=routing.row_of_slot, rq=rq, rs=rs, u=u, q2=q2, s2=s2, d=d, out=out)


def moe_inputs(M, seed, dropped):
    rng = np.random.default_rng(seed)
    ids = np.argsort(rng.random((M, E)), axis=1)[:, :TOPK].astype(np.int32)
    ids[rng.random((M, TOPK)) < dropped] = -1
    w = rng.random((M, TOPK)).astype(np.float32)
    return synth.activations(M, HID, seed), synth.activations(M, HID, seed + 1), ids, w


@pytest.mark.parametrize("M", [1, 4, 37, 200])
@pytest.mark.parametrize("dropped", [0.0, 0.3])
def test_moe_block(ops, M, dropped):
    announce(f"moe block M={M} dropped={dropped}")
    wg, wd, gate_up, down = moe_weights(ops)
    x, res, ids, w = moe_inputs(M, 50 + M, dropped)
    g = synth.normal_bf16((HID,), 9)
    t = moe_block(ops, ops.RMSNorm(dev_bf16(g), EPS), gate_up, down, dev_bf16(x), dev_bf16(res), torch.from_numpy(ids).cuda(),
                  torch.from_numpy(w).cuda())
    torch.cuda.synchronize()
    h64, y64 = block.rms_norm(f64(x), f64(res), f64(g), EPS)
    assert_bf16(t["y"], y64, "norm")
    assert_codes(t["q"], t["s"], y64, "e4m3", "norm to e4m3")
    off, row = block.route(ids, E)
    assert np.array_equal(t["off"].cpu().numpy(), off) and np.array_equal(t["row"].cpu().numpy(), row)
    n = off[-1]
    q, s = t["q"].cpu().numpy(), t["s"].cpu().numpy()
    rq, rs = t["rq"].cpu().numpy()[:n], t["rs"].cpu().numpy()[:n]
    assert np.array_equal(rq, block.gather(q, row, np.zeros((M * TOPK, HID), np.uint8))[:n])
    assert np.array_equal(rs, block.gather(s, row, np.zeros(M * TOPK, np.float32))[:n])
    dec = lambda c, sc: f8.e4m3_decode(c).astype(np.float64) * sc.astype(np.float64)[:, None]

    def grouped(a, ws):
        return np.concatenate([a[off[e]:off[e + 1]] @ dequant(ws[e]) for e in range(E)])
    if n:
        assert_close_rms(host_bits16(t["u"])[:n], grouped(dec(rq, rs), wg), what="grouped gate_up")
        u = host(t["u"])[:n]
        assert_codes(t["q2"][:n], t["s2"][:n], block.swiglu(u), "e4m3", "swiglu", gate_floor(u))
        a2 = dec(t["q2"].cpu().numpy()[:n], t["s2"].cpu().numpy()[:n])
        assert_close_rms(host_bits16(t["d"])[:n], grouped(a2, wd), what="grouped down")
    d = host(t["d"])
    d[n:] = 0
    w64 = np.where(row >= 0, w, 0).astype(np.float64)
    ref = block.combine(d, row, w64, host(t["h"]))
    size = block.combine(np.abs(d), row, w64, np.abs(host(t["h"])))
    err = np.abs(host(t["out"]) - ref)
    # half a bf16 step, and TOPK + 1 fp32 roundings of the terms
    assert (err <= 2.0 ** -8 * np.abs(ref) * (1 + 2.0 ** -8) + (TOPK + 1) * 2.0 ** -23 * size).all()


@pytest.mark.parametrize("M", [1, 20, 600])
def test_block_in_a_graph(ops, M):
    """Captured once, replayed on new inputs, with eager work between the replays:
    every replay gives the eager call's bits (600 tokens: the separate sort)."""
    announce(f"moe block in a graph M={M}")
    _, _, gate_up, down = moe_weights(ops)
    norm = ops.RMSNorm(dev_bf16(synth.normal_bf16((HID,), 9)), EPS)
    lin = ops.W4A16Linear(ops.Int4G128Weight.from_bf16(dev_bf16(synth.weights(HID, HID, 2))),
                          dev_bf16(synth.normal_bf16((HID,), 5)), "gelu")

    def load(seed):
        x, res, ids, w = moe_inputs(M, seed, 0.2)
        return [dev_bf16(x), dev_bf16(res), torch.from_numpy(ids).cuda(), torch.from_numpy(w).cuda()]

    def step(x, res, ids, w):
        out = moe_block(ops, norm, gate_up, down, x, res, ids, w)["out"]
        return out, lin(out, residual=res)

    held = load(100)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(*held)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step(*held)
    for seed in (101, 102, 103, 101):
        new = load(seed)
        for a, b in zip(held, new):
            a.copy_(b)
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in outs]
        want = step(*new)                                     # eager work between the replays
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b), f"replay on inputs {seed}"


def test_two_streams(ops):
    """Two blocks under way on two streams give what they give alone."""
    announce("two streams")
    norm = ops.RMSNorm(dev_bf16(synth.normal_bf16((HID,), 9)), EPS)
    wg = [moe_weights(ops)[2:] for _ in range(2)]             # each stream's own weights and workspaces
    sets, alone = [], []
    for i, M in enumerate((300, 700)):
        x, res, ids, w = moe_inputs(M, 200 + i, 0.1)
        sets.append([dev_bf16(x), dev_bf16(res), torch.from_numpy(ids).cuda(), torch.from_numpy(w).cuda()])
        alone.append(moe_block(ops, norm, *wg[i], *sets[i])["out"].clone())
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        outs = [None, None]
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                outs[i] = moe_block(ops, norm, *wg[i], *sets[i])["out"]
        torch.cuda.synchronize()
        for a, b in zip(outs, alone):
            assert torch.equal(a, b)


def test_stream_argument(ops):
    """An explicit stream is the one the work runs on."""
    announce("explicit stream")
    x = dev_bf16(synth.activations(4, 4096, 1))
    norm = ops.RMSNorm(dev_bf16(synth.normal_bf16((4096,), 9)), EPS)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    want, _ = norm(x)
    got, _ = norm(x, stream=st)
    st.synchronize()
    torch.cuda.synchronize()
    assert torch.equal(got, want)


def test_memory_of_an_explicit_stream(ops):
    """A helper's workspace, freed when the helper returns, is not handed to the
    current stream while the given stream still has to use it."""
    announce("workspace of an explicit stream")
    B, k, n_exp = 4096, 8, 64
    rng = np.random.default_rng(3)
    ids_h = rng.integers(0, n_exp, (B, k)).astype(np.int32)
    ids = torch.from_numpy(ids_h).cuda()
    need = ops.moe_dispatch_workspace_bytes(B, k, n_exp)
    assert need > 0
    a = torch.randn((4096, 4096), device="cuda:0")
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(st):
        for _ in range(8):                                    # a few milliseconds ahead of the dispatch
            a = torch.sin(a @ a)
    r, _, _ = ops.MoeRouting.dispatch(ids, n_exp, stream=st)
    spoil = [torch.full((need,), 0x7F, dtype=torch.uint8, device="cuda:0") for _ in range(64)]
    torch.cuda.synchronize()
    off, row = r.offsets.cpu().numpy(), r.row_of_slot.cpu().numpy()
    del spoil
    order = np.argsort(ids_h.reshape(-1), kind="stable")
    want = np.empty(B * k, np.int32)
    want[order] = np.arange(B * k)
    assert np.array_equal(row.reshape(-1), want)
    assert np.array_equal(off, np.searchsorted(np.sort(ids_h.reshape(-1)), np.arange(n_exp + 1)))
