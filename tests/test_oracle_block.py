"""Pins of oracle/block.py: hand-worked values, torch's own fp64 functions and
finite differences."""
import math

import numpy as np
import torch

from oracle import block


def test_rms_norm_by_hand():
    h, y = block.rms_norm(np.array([[3.0, 4.0]]), np.array([[0.0, -8.0]]), np.array([2.0, 1.0]), 0.0)
    assert np.array_equal(h, [[3.0, -4.0]])
    assert np.allclose(y, [[3 / math.sqrt(12.5) * 2, -4 / math.sqrt(12.5)]], rtol=1e-15)


def test_functions_against_torch_fp64():
    x = torch.linspace(-40, 40, 2001, dtype=torch.float64)
    F = torch.nn.functional
    for name, ref in (("relu", F.relu(x)), ("silu", F.silu(x)), ("gelu", F.gelu(x)),
                      ("gelu_tanh", F.gelu(x, approximate="tanh")), ("none", x)):
        got = block.activation(x.numpy(), name)
        assert np.allclose(got, ref.numpy(), rtol=1e-9, atol=1e-12), name
    g = torch.randn(3, 16, dtype=torch.float64)
    assert np.allclose(block.swiglu(g.numpy()), (F.silu(g[:, :8]) * g[:, 8:]).numpy(), rtol=1e-13)
    assert np.isfinite(block.silu(np.array([-1e4, 1e4]))).all()
    w = torch.randn(16, dtype=torch.float64)
    assert np.allclose(block.rms_norm(g.numpy(), None, w.numpy(), 1e-5)[1], F.rms_norm(g, (16,), w, 1e-5).numpy())


def test_routing_by_hand():
    ids = np.array([[2, 0], [-1, 2], [0, 3]])
    offsets, row = block.route(ids, 3)
    assert offsets.tolist() == [0, 2, 2, 4]
    assert row.tolist() == [[2, 0], [-1, 3], [1, -1]]
    rows = np.arange(12.0).reshape(6, 2)
    y = block.combine(rows, row, np.full((3, 2), 0.5), np.ones((3, 2)))
    assert y.tolist() == [[1 + 0.5 * (4 + 0), 1 + 0.5 * (5 + 1)], [1 + 3.0, 1 + 3.5], [1 + 1.0, 1 + 1.5]]
    assert block.gather(np.array([[1.0], [2.0], [3.0]]), row, np.full((6, 1), 9.0)).ravel().tolist() == [1, 3, 1, 2, 9, 9]


def test_combine_gradient_against_differences():
    rng = np.random.default_rng(0)
    ids = rng.integers(-1, 4, (5, 3))
    _, row = block.route(ids, 4)
    rows, w, dy = rng.standard_normal((15, 4)), rng.random((5, 3)), rng.standard_normal((5, 4))
    drows, dw = block.combine_backward(dy, rows, row, w)
    loss = lambda r, v: (block.combine(r, row, v, None) * dy).sum()
    for i in np.ndindex(rows.shape):
        e = np.zeros_like(rows)
        e[i] = 0.5
        assert abs(loss(rows + e, w) - loss(rows - e, w) - drows[i]) < 1e-12
    for i in np.ndindex(w.shape):
        e = np.zeros_like(w)
        e[i] = 0.5
        assert abs(loss(rows, w + e) - loss(rows, w - e) - dw[i]) < 1e-12
