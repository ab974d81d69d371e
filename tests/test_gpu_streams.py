"""Work on a stream that the caller gives: what it reads, clears and keeps is ordered
on that stream, whatever the current stream is busy with.
"""
import numpy as np
import pytest
import torch

from gpu_helpers import announce, dev_bf16
from weight_only_quantized_w4a16_amd import synth

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ops():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    from weight_only_quantized_w4a16_amd import ops as _ops
    return _ops


class Busy:
    """A few milliseconds of work on the current stream."""

    def __init__(self):
        self.a = torch.randn((4096, 4096), device="cuda:0")
        self.a @ self.a                                       # the library's own preparations

    def __call__(self):
        for _ in range(8):
            self.a = torch.sin(self.a @ self.a)


# dense products whose plans split K (workspaces with counters), with M rows that grow
SPLIT = [(16, 1024, 14336), (100, 4096, 4096)]


def products(ops, N, K):
    """name -> a function that makes a new helper and returns its call."""
    w = dev_bf16(synth.weights(K, N, seed=3))
    w4, w8, wi = ops.Int4G128Weight.from_bf16(w), ops.Fp8Weight.from_bf16(w), ops.Int8Weight.from_bf16(w)
    bias = dev_bf16(synth.normal_bf16((N,), 2))
    return {
        "w4a16": lambda: ops.W4A16Linear(w4),
        "w4a16 epilogue": lambda: ops.W4A16Linear(w4, bias, "gelu"),
        "w8a8 fp8": lambda: ops.W8A8Fp8Linear(w8),
        "w8a8 int8": lambda: ops.W8A8Int8Linear(wi),
        "w4a8": lambda: ops.W4A8Linear(w4),
    }


@pytest.mark.parametrize("M,N,K", SPLIT)
def test_first_call_on_another_stream(ops, M, N, K):
    """The first call brings its workspace: its clearing must not wait behind the current stream's work."""
    announce(f"first call on another stream M={M} N={N} K={K}")
    assert not ops.w4a16_kernel_for(M, N, K).endswith("S=1")
    a = dev_bf16(synth.activations(M, K, seed=1))
    makers = products(ops, N, K)
    want = {name: make()(a) for name, make in makers.items()}
    busy, st = Busy(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for name, make in makers.items():
        lin = make()
        busy()
        got = lin(a, stream=st)
        again = lin(a, stream=st)
        st.synchronize()
        assert torch.equal(got, want[name]) and torch.equal(again, want[name]), name
        torch.cuda.synchronize()


def test_growing_on_another_stream(ops):
    """A workspace that a call outgrows is not handed out while the given stream still uses it."""
    announce("workspace outgrown on another stream")
    N, K = 4096, 4096
    small, large = (dev_bf16(synth.activations(M, K, seed=M)) for M in (70, 100))
    need = ops.w4a16_workspace_bytes(70, N, K)
    assert 0 < need < ops.w4a16_workspace_bytes(100, N, K)
    make = products(ops, N, K)["w4a16 epilogue"]
    want = make()(small), make()(large)
    busy, st = Busy(), torch.cuda.Stream()
    for _ in range(3):
        lin = make()
        first = lin(small)                                    # the workspace belongs to the current stream
        torch.cuda.synchronize()
        with torch.cuda.stream(st):
            busy()
        got = lin(small, stream=st), lin(large, stream=st)
        spoil = [torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda:0") for _ in range(16)]
        torch.cuda.synchronize()
        assert torch.equal(first, want[0]) and torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        del spoil


def test_work_follows_the_given_stream(ops):
    """Inputs that an earlier piece of work on the given stream writes are the ones that a call there reads."""
    announce("order on the given stream")
    Mx, Kx = 64, 4096
    old, new = dev_bf16(synth.activations(Mx, Kx, 1)), dev_bf16(synth.activations(Mx, Kx, 2))
    w = dev_bf16(synth.normal_bf16((Kx,), 9))
    ids_old = torch.zeros((Mx, 4), dtype=torch.int32, device="cuda:0")
    ids_new = torch.from_numpy(np.random.default_rng(0).integers(0, 8, (Mx, 4)).astype(np.int32)).cuda()
    norm = ops.RMSNorm(w)
    y = torch.empty((Mx, Kx), dtype=torch.bfloat16, device="cuda:0")
    q, s = torch.empty((Mx, Kx), dtype=torch.uint8, device="cuda:0"), torch.empty(Mx, device="cuda:0")
    half = torch.empty((Mx, Kx // 2), dtype=torch.bfloat16, device="cuda:0")

    def raw(call, out):
        def f(x, ids, stream):
            out.zero_() if stream is None else None
            call(x, stream)
            return out
        return f
    calls = {
        "norm": lambda x, ids, st: norm(x, stream=st)[0],
        "norm quantized": lambda x, ids, st: norm.quantized(x, stream=st)[0],
        "gated_silu": lambda x, ids, st: ops.gated_silu(x, stream=st),
        "gated_silu_quantized": lambda x, ids, st: ops.gated_silu_quantized(x, "int8", stream=st)[0],
        "dispatch": lambda x, ids, st: ops.MoeRouting.dispatch(ids, 8, x, stream=st)[1],
        "rms_norm": raw(lambda x, st: ops.rms_norm(x, None, w, 1e-5, Mx, Kx, None, y, stream=st), y),
        "rms_norm_quant": raw(lambda x, st: ops.rms_norm_quant(x, None, w, 1e-5, Mx, Kx, None, None, q, s, stream=st), q),
        "swiglu": raw(lambda x, st: ops.swiglu(x, Mx, Kx // 2, half, stream=st), half),
    }
    busy, st = Busy(), torch.cuda.Stream()
    for name, f in calls.items():
        want = f(new, ids_new, None).clone()
        x, ids = old.clone(), ids_old.clone()
        torch.cuda.synchronize()
        with torch.cuda.stream(st):
            busy()
            x.copy_(new)
            ids.copy_(ids_new)
        got = f(x, ids, st)
        assert not st.query(), "the work ahead was over too soon to show an order"
        st.synchronize()
        assert torch.equal(got, want), name
        torch.cuda.synchronize()


@pytest.mark.parametrize("M,N,K", SPLIT)
def test_workspace_of_a_captured_first_call(ops, M, N, K):
    """Captured before any eager call, then used eagerly, replayed, outgrown and replayed again."""
    announce(f"captured first call M={M} N={N} K={K}")
    a, b = (dev_bf16(synth.activations(M, K, seed=s)) for s in (1, 2))
    more = dev_bf16(synth.activations(128, K, seed=3))
    for name, make in products(ops, N, K).items():
        want_a, want_b, want_more = make()(a), make()(b), make()(more)
        torch.cuda.synchronize()
        lin, held = make(), a.clone()
        graphs, outs = [], []
        for _ in range(2):                                    # the second with the eager calls' workspace
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                outs.append(lin(held))
            graphs.append(graph)
            assert torch.equal(lin(b), want_b), name
        assert torch.equal(lin(more), want_more), name        # may outgrow it
        spoil = [torch.full((1 << 20,), 0xFF, dtype=torch.uint8, device="cuda:0") for _ in range(32)]
        for turn in range(4):
            held.copy_((a, b)[turn % 2])
            for graph, out in zip(graphs, outs):
                graph.replay()
                torch.cuda.synchronize()
                assert torch.equal(out, (want_a, want_b)[turn % 2]), f"{name} replay {turn}"
                assert torch.equal(lin(b), want_b), name
        del spoil
