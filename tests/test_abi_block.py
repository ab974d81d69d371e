"""The operators between two products reject invalid arguments on the host,
before anything is launched.

Runs without a GPU: every call fails validation (or has nothing to do), so the
pointers are never dereferenced.
"""
import ctypes
import os

import pytest

from conftest import ROOT

LIB = os.path.join(ROOT, "weight_only_quantized_w4a16_amd", "libqgemm.so")
QG_OK, QG_ERR_NULL, QG_ERR_SHAPE, QG_ERR_ALIGN, QG_ERR_WORKSPACE, QG_ERR_HIP = range(6)
FAKE = 0x4000000

pytestmark = pytest.mark.skipif(not os.path.exists(LIB), reason="libqgemm.so not built")


@pytest.fixture(scope="module")
def ops():
    from weight_only_quantized_w4a16_amd import ops as _ops
    return _ops


def call(ops, name, defaults, **changed):
    args = dict(defaults, **changed)
    return getattr(ops._lib, name)(*args.values(), None)


NORM = dict(x=FAKE, r=FAKE, w=FAKE, eps=1e-5, M=2, K=64, h=FAKE, y=FAKE)
QUANT = dict(NORM, q=FAKE, s=FAKE)
BAD_ROWS = [dict(M=-1), dict(K=0), dict(K=-8), dict(K=12), dict(K=(1 << 20) + 8), dict(M=1 << 22),
            dict(M=(1 << 22) - 1, K=8200)]


@pytest.mark.parametrize("changed", BAD_ROWS + [dict(eps=e) for e in
                                                (0.0, -1e-5, 1e-39, float("inf"), float("nan"))])
def test_norm_shapes(ops, changed):
    assert call(ops, "rms_norm", NORM, **changed) == QG_ERR_SHAPE
    assert call(ops, "rms_norm_quant", QUANT, **changed) == QG_ERR_SHAPE
    assert call(ops, "rms_norm_quant_int8", QUANT, **changed) == QG_ERR_SHAPE


def test_norm_pointers(ops):
    for name, base in (("rms_norm", NORM), ("rms_norm_quant", QUANT), ("rms_norm_quant_int8", QUANT)):
        need = ("x", "w", "y") if name == "rms_norm" else ("x", "w", "q", "s")
        for p in need:
            assert call(ops, name, base, **{p: None}) == QG_ERR_NULL, (name, p)
        for p in base:
            if p not in ("eps", "M", "K"):
                assert call(ops, name, base, **{p: FAKE + 2}) == QG_ERR_ALIGN, (name, p)
        assert call(ops, name, base, M=0, x=None) == QG_OK


def test_swiglu_refusals(ops):
    plain = dict(gu=FAKE, M=2, I=64, y=FAKE)
    quant = dict(gu=FAKE, M=2, I=64, q=FAKE, s=FAKE)
    for name, base in (("swiglu", plain), ("swiglu_quant", quant), ("swiglu_quant_int8", quant)):
        for changed in BAD_ROWS:
            assert call(ops, name, base, **{{"K": "I"}.get(k, k): v for k, v in changed.items()}) == QG_ERR_SHAPE
        for p in set(base) - {"M", "I"}:
            assert call(ops, name, base, **{p: None}) == QG_ERR_NULL, (name, p)
            assert call(ops, name, base, **{p: FAKE + 2}) == QG_ERR_ALIGN, (name, p)
        assert call(ops, name, base, M=0, gu=None) == QG_OK


DISPATCH = dict(ids=FAKE, rows=FAKE, rs=FAKE, B=4, k=2, E=8, width=64, offsets=FAKE, row=FAKE, out=FAKE, so=FAKE,
                ws=FAKE, wsb=1 << 20)
GATHER = dict(rows=FAKE, rs=FAKE, row=FAKE, B=4, k=2, width=64, out=FAKE, so=FAKE)
COMBINE = dict(rows=FAKE, row=FAKE, w=FAKE, res=FAKE, B=4, k=2, K=64, y=FAKE)
BACKWARD = dict(dy=FAKE, rows=FAKE, row=FAKE, w=FAKE, B=4, k=2, K=64, drows=FAKE, dw=FAKE)
BAD_SLOTS = [dict(B=-1), dict(B=1 << 22), dict(k=0), dict(k=1025), dict(B=(1 << 22) - 1, k=8)]


def test_moe_shapes(ops):
    for changed in BAD_SLOTS:
        for name, base in (("moe_dispatch", DISPATCH), ("moe_gather", GATHER), ("moe_combine", COMBINE),
                           ("moe_combine_backward", BACKWARD)):
            assert call(ops, name, base, **changed) == QG_ERR_SHAPE, (name, changed)
    for E in (0, -1, 1025):
        assert call(ops, "moe_dispatch", DISPATCH, E=E) == QG_ERR_SHAPE
        assert ops.moe_dispatch_workspace_bytes(4, 2, E) == 0
    for width in (0, -8, 4, 12, (1 << 21) + 8):
        assert call(ops, "moe_dispatch", DISPATCH, width=width) == QG_ERR_SHAPE
        assert call(ops, "moe_gather", GATHER, width=width) == QG_ERR_SHAPE
    for K in (0, -8, 12, (1 << 20) + 8):
        assert call(ops, "moe_combine", COMBINE, K=K) == QG_ERR_SHAPE
        assert call(ops, "moe_combine_backward", BACKWARD, K=K) == QG_ERR_SHAPE
    # too many workgroups: 2^22 - 1 tokens of 5 parts
    assert call(ops, "moe_combine", COMBINE, B=(1 << 22) - 1, K=8 * 256 * 4 + 8) == QG_ERR_SHAPE
    assert call(ops, "moe_gather", GATHER, B=(1 << 22) - 1, k=1, width=8 * 256 * 4 + 8) == QG_ERR_SHAPE


def test_moe_pointers(ops):
    for p in ("ids", "offsets", "row", "ws"):
        assert call(ops, "moe_dispatch", DISPATCH, B=65536, **{p: None}) == QG_ERR_NULL, p
    # rows and their destination come together, and so do scales; scales need rows
    for changed in (dict(rows=None), dict(out=None), dict(rs=None), dict(so=None), dict(rows=None, out=None)):
        assert call(ops, "moe_dispatch", DISPATCH, **changed) == QG_ERR_NULL, changed
    assert call(ops, "moe_dispatch", DISPATCH, B=65536, wsb=3) == QG_ERR_WORKSPACE
    assert call(ops, "moe_dispatch", DISPATCH, B=0, offsets=None) == QG_ERR_NULL
    for p in ("rows", "row", "out", "rs", "so"):
        assert call(ops, "moe_gather", GATHER, **{p: None}) == QG_ERR_NULL, p
    for p in ("rows", "row", "y"):
        assert call(ops, "moe_combine", COMBINE, **{p: None}) == QG_ERR_NULL, p
    for p in ("dy", "row", "rows"):
        assert call(ops, "moe_combine_backward", BACKWARD, **{p: None}) == QG_ERR_NULL, p
    assert call(ops, "moe_combine_backward", BACKWARD, drows=None, dw=None) == QG_ERR_NULL
    for name, base in (("moe_dispatch", DISPATCH), ("moe_gather", GATHER), ("moe_combine", COMBINE),
                       ("moe_combine_backward", BACKWARD)):
        for p, v in base.items():
            if v == FAKE and not (name == "moe_dispatch" and p == "ws"):
                assert call(ops, name, base, **{p: FAKE + 2}) == QG_ERR_ALIGN, (name, p)
    assert call(ops, "moe_dispatch", DISPATCH, B=65536, ws=FAKE + 2) == QG_ERR_ALIGN
    for name, base in (("moe_gather", GATHER), ("moe_combine", COMBINE), ("moe_combine_backward", BACKWARD)):
        assert call(ops, name, base, B=0, row=None) == QG_OK


def test_binding_refuses_host_tensors(ops):
    import torch
    x = torch.zeros((2, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="on the GPU"):
        ops.rms_norm(x, None, x[0], 1e-5, 2, 64, None, x)
    with pytest.raises(ValueError):
        ops.moe_combine(None, None, None, None, 0, 1, 8, None)


EPILOGUE = dict(a=FAKE, w=FAKE, sc=FAKE, b=FAKE, act=1, res=FAKE, y=FAKE, M=4, N=64, K=256, ws=None, wsb=0)


def test_epilogue_refusals(ops):
    name = "qgemm_w4a16_epilogue"
    for changed in (dict(M=-1), dict(N=8), dict(K=64), dict(act=-1), dict(act=5), dict(M=1 << 25)):
        assert call(ops, name, EPILOGUE, **changed) == QG_ERR_SHAPE, changed
    for p in ("a", "w", "sc", "y"):
        assert call(ops, name, EPILOGUE, **{p: None}) == QG_ERR_NULL, p
    for p in ("a", "w", "sc", "b", "res", "y"):
        assert call(ops, name, EPILOGUE, **{p: FAKE + 2}) == QG_ERR_ALIGN, p
    assert call(ops, name, EPILOGUE, M=100) == QG_ERR_NULL            # needs a workspace
    assert call(ops, name, EPILOGUE, M=100, ws=FAKE, wsb=16) == QG_ERR_WORKSPACE
    assert call(ops, name, EPILOGUE, M=100, ws=FAKE + 4, wsb=1 << 30) == QG_ERR_ALIGN
    assert call(ops, name, EPILOGUE, M=0, a=None) == QG_OK


def test_activation_names(ops):
    import re
    text = open(os.path.join(ROOT, "include", "qgemm.h")).read()
    codes = {n.lower(): int(v) for n, v in re.findall(r"QG_ACT_(\w+) = (\d+)", text)}
    assert codes == ops.ACTIVATIONS
    from oracle import block
    assert set(block.EPILOGUE_ACTIVATIONS) == set(codes)


def test_binding_refuses_wrong_arguments(ops):
    with pytest.raises(TypeError, match="tensor or None"):
        ops.rms_norm("x", None, None, 1e-5, 2, 64, None, None)
    with pytest.raises(TypeError):
        ops.swiglu(None, 2.5, 64, None)
    with pytest.raises(OverflowError):
        ops.swiglu(None, 2 ** 40, 64, None)
    with pytest.raises((OverflowError, ValueError)):
        ops.moe_dispatch(None, None, None, 1, 1, 1, 0, None, None, None, None, None, -1)
    with pytest.raises(ValueError, match="no tensor"):
        ops.swiglu(None, 2, 64, None)
    with pytest.raises(ValueError, match="activation"):
        ops.qgemm_w4a16_epilogue(None, None, None, None, "tanh", None, None, 1, 16, 128)
