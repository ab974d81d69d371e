"""CPU oracle of the operators between two products of a decoder block, in fp64
(test infrastructure only): residual + root-mean-square norm, the gated unit,
per-token codes of their outputs, expert routing with its gradient, and the
epilogue of a product (bias, activation, residual).

Inputs are float64 arrays of the values the library receives.
"""
import math

import numpy as np

EPILOGUE_ACTIVATIONS = ("none", "relu", "gelu", "gelu_tanh", "silu")


def rms_norm(x, residual, weight, eps):
    """(h, y): h = x + residual, y = h / sqrt(mean(h^2) + eps) * weight."""
    h = x if residual is None else x + residual
    return h, h / np.sqrt(np.mean(h * h, axis=1, keepdims=True) + eps) * weight


def silu(g):
    with np.errstate(over="ignore"):
        return np.where(g >= 0, g / (1 + np.exp(-np.abs(g))), g * np.exp(-np.abs(g)) / (1 + np.exp(-np.abs(g))))


def swiglu(gate_up):
    n = gate_up.shape[1] // 2
    return silu(gate_up[:, :n]) * gate_up[:, n:]


def route(expert_ids, E):
    """(offsets [E + 1], row_of_slot like expert_ids): slots in order inside an
    expert, experts ascending, -1 for an id outside [0, E)."""
    flat = np.asarray(expert_ids).reshape(-1)
    row = np.full(flat.shape, -1, np.int32)
    offsets = np.zeros(E + 1, np.int32)
    at = 0
    for e in range(E):
        for s in np.nonzero(flat == e)[0]:
            row[s] = at
            at += 1
        offsets[e + 1] = at
    return offsets, row.reshape(np.shape(expert_ids))


def gather(rows, row_of_slot, out):
    """out with every token's row at its routed rows (other rows kept)."""
    out = out.copy()
    for b, j in zip(*np.nonzero(row_of_slot >= 0)):
        out[row_of_slot[b, j]] = rows[b]
    return out


def combine(rows, row_of_slot, weights, residual):
    B, k = row_of_slot.shape
    y = np.zeros((B, rows.shape[1])) if residual is None else residual.copy()
    for b, j in zip(*np.nonzero(row_of_slot >= 0)):
        y[b] += (1.0 if weights is None else weights[b, j]) * rows[row_of_slot[b, j]]
    return y


def combine_backward(dy, rows, row_of_slot, weights):
    """(drows, dweights); drows is 0 for a row of no slot."""
    drows = np.zeros_like(rows)
    dw = np.zeros(row_of_slot.shape)
    for b, j in zip(*np.nonzero(row_of_slot >= 0)):
        r = row_of_slot[b, j]
        drows[r] = (1.0 if weights is None else weights[b, j]) * dy[b]
        dw[b, j] = dy[b] @ rows[r]
    return drows, dw


_erfc = np.vectorize(math.erfc, otypes=[np.float64])


def activation(x, name):
    if name == "none":
        return x
    if name == "relu":
        return np.maximum(x, 0.0)
    if name == "silu":
        return silu(x)
    if name == "gelu":
        return x * 0.5 * _erfc(-x / math.sqrt(2.0))
    if name == "gelu_tanh":
        # 0.5 x (1 + tanh(z)) = x sigmoid(2 z)
        z = 2 * math.sqrt(2 / math.pi) * (x + 0.044715 * x ** 3)
        e = np.exp(-np.abs(z))
        return x * np.where(z >= 0, 1 / (1 + e), e / (1 + e))
    raise ValueError(name)


def epilogue(product, bias, name, residual):
    y = activation(product if bias is None else product + bias, name)
    return y if residual is None else y + residual
