"""MoeRouting's helpers inside torch's autograd: the gradients that
moe_combine_backward and moe_combine compute arrive at the leaves.
"""
import numpy as np
import pytest
import torch

from gpu_helpers import announce, dev_bf16, host_bits16
from oracle import block
from oracle.bf16 import bf16_bits_to_f32
from weight_only_quantized_w4a16_amd import synth

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ops():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    from weight_only_quantized_w4a16_amd import ops as _ops
    return _ops


def f64(bits):
    return bf16_bits_to_f32(bits).astype(np.float64)


def inputs(B, k, E, K, seed, dropped=0.2):
    rng = np.random.default_rng(seed)
    ids = rng.integers(0, E, (B, k)).astype(np.int32)
    ids[rng.random((B, k)) < dropped] = -1
    w = torch.from_numpy(rng.random((B, k)).astype(np.float32)).cuda()
    x, res, dy = (dev_bf16(synth.normal_bf16((B, K), seed + i)) for i in range(3))
    return torch.from_numpy(ids).cuda(), w, x, res, dy


@pytest.mark.parametrize("B,k,E,K", [(1, 1, 1, 8), (5, 3, 4, 64), (33, 8, 16, 520), (700, 2, 60, 1032)])
def test_gradients(ops, B, k, E, K):
    """Of dispatch -> combine, against the explicit calls and the oracle.  Where the routed rows are a leaf, rows of
    no slot get zeros."""
    announce(f"combine autograd B={B} k={k} E={E} K={K}")
    ids, w, x, res, dy = inputs(B, k, E, K, 3)
    r0, rows0, _ = ops.MoeRouting.dispatch(ids, E, x)
    y0 = r0.combine(rows0, w, res)
    drows0, dw0 = r0.combine_backward(dy, rows0, w)
    dx0 = r0.combine(drows0)

    leaves = [t.clone().requires_grad_() for t in (x, w, res)]
    r, rows, _ = ops.MoeRouting.dispatch(ids, E, leaves[0])
    y = r.combine(rows, leaves[1], leaves[2])
    y.backward(dy)
    torch.cuda.synchronize()
    n = int(r0.offsets[-1])
    assert torch.equal(r.offsets, r0.offsets) and torch.equal(r.row_of_slot, r0.row_of_slot)
    assert torch.equal(rows[:n], rows0[:n]) and torch.equal(y, y0)
    assert torch.equal(leaves[0].grad, dx0) and torch.equal(leaves[1].grad, dw0) and torch.equal(leaves[2].grad, dy)

    leaf = torch.where(torch.arange(B * k, device="cuda:0")[:, None] < n, rows0, torch.full_like(rows0, float("nan")))
    leaf.requires_grad_()
    r0.combine(leaf, w).backward(dy)
    torch.cuda.synchronize()
    assert torch.equal(leaf.grad[:n], drows0[:n]) and not bool(leaf.grad[n:].any())

    # the oracle on the same values: a weight's gradient is a difference of the loss, which is linear in it
    row = r0.row_of_slot.cpu().numpy()
    routed = f64(host_bits16(rows0))
    routed[n:] = 0
    dw64 = block.combine_backward(f64(host_bits16(dy)), routed, row, w.cpu().numpy().astype(np.float64))[1]
    size = block.combine_backward(np.abs(f64(host_bits16(dy))), np.abs(routed), row, None)[1]
    got = leaves[1].grad.cpu().numpy().astype(np.float64)
    assert (np.abs(got - dw64) <= (8 * -(-K // 2048) + 11) * 2.0 ** -24 * size + 2.0 ** -149).all()


def test_against_differences(ops):
    """The gradient of sum(dy * combine(gather(x), w) + dy * residual) against central differences of the oracle."""
    announce("combine autograd against differences")
    B, k, E, K = 4, 3, 5, 16
    ids, w, x, res, dy = inputs(B, k, E, K, 11)
    leaves = [t.clone().requires_grad_() for t in (x, w, res)]
    r, _, _ = ops.MoeRouting.dispatch(ids, E)
    rows, _ = r.gather(leaves[0])
    (r.combine(rows, leaves[1], leaves[2]).float() * dy.float()).sum().backward()
    torch.cuda.synchronize()
    row, d = r.row_of_slot.cpu().numpy(), f64(host_bits16(dy))
    X, W, R = f64(host_bits16(x)), w.cpu().numpy().astype(np.float64), f64(host_bits16(res))
    loss = lambda X, W, R: float((block.combine(block.gather(X, row, np.zeros((B * k, K))), row, W, R) * d).sum())
    for leaf, at in zip(leaves, (X, W, R)):
        grad = leaf.grad.float().cpu().numpy()
        for i in np.ndindex(*at.shape):
            keep = at[i]
            at[i] = keep + 0.5
            up = loss(X, W, R)
            at[i] = keep - 0.5
            num = up - loss(X, W, R)
            at[i] = keep
            # each of k terms and their sum rounded to bf16 at most
            assert abs(num - grad[i]) <= (k + 1) * 2.0 ** -8 * np.abs(d).max() + 1e-9, (i, num, grad[i])


def test_without_gradients(ops):
    """No graph under no_grad, nor without a leaf; what has no gradient is refused, not cut off."""
    announce("combine autograd off")
    ids, w, x, res, dy = inputs(6, 2, 4, 64, 5, dropped=0.0)
    wl = w.clone().requires_grad_()
    r, rows, _ = ops.MoeRouting.dispatch(ids, 4, x)
    assert not rows.requires_grad and not r.combine(rows, w, res).requires_grad
    with torch.no_grad():
        assert not r.combine(rows, wl, res).requires_grad
    y = r.combine(rows, wl, res)
    assert y.requires_grad
    with pytest.raises(RuntimeError, match="out="):
        r.combine(rows, wl, res, out=torch.empty_like(x))
    with pytest.raises(TypeError, match="bf16"):
        ops.MoeRouting.dispatch(ids, 4, x.float().requires_grad_())
    # an expanded gradient (that of a sum)
    y.sum().backward()
    torch.cuda.synchronize()
    want = r.combine_backward(torch.ones_like(x), rows, w)[1]
    assert torch.equal(wl.grad, want)


def test_on_a_stream_and_twice(ops):
    """On an explicit stream; two graphs over the same leaf add up."""
    announce("combine autograd on a stream")
    ids, w, x, res, dy = inputs(40, 4, 8, 256, 7)
    r, rows, _ = ops.MoeRouting.dispatch(ids, 8, x)
    want = r.combine_backward(dy, rows, w)[1]
    wl = w.clone().requires_grad_()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    y1 = r.combine(rows, wl, res, stream=st)
    torch.cuda.current_stream().wait_stream(st)
    y2 = r.combine(rows, wl)
    y1.backward(dy)
    y2.backward(dy)
    torch.cuda.synchronize()
    assert torch.equal(wl.grad, want + want)


def test_captured_step(ops):
    """A training step of the router's weights captured in a graph, replayed on new inputs: the eager bits."""
    announce("combine autograd in a graph")
    B, k, E, K = 24, 4, 8, 256
    ids, w, x, res, dy = inputs(B, k, E, K, 13)

    def step(wl):
        r, rows, _ = ops.MoeRouting.dispatch(ids, E, x)
        return torch.autograd.grad(r.combine(rows, wl, res), wl, dy)[0]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(w.clone().requires_grad_())
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(w.detach().requires_grad_())
    for seed in (13, 14, 15):
        for held, new in zip((ids, w, x, res, dy), inputs(B, k, E, K, seed)):
            held.copy_(new)
        graph.replay()
        torch.cuda.synchronize()
        kept = got.clone()
        want = step(w.clone().requires_grad_())               # eager work between the replays
        torch.cuda.synchronize()
        assert torch.equal(kept, want), seed
