"""The tensor-level helpers allocate, clear and launch on the stream they are given.

Runs without a GPU: torch's allocations and the raw entry points are replaced by
recorders of the stream that is current when they are called.
"""
import contextlib
import os
import types
import weakref

import pytest
import torch

from conftest import ROOT

LIB = os.path.join(ROOT, "weight_only_quantized_w4a16_amd", "libqgemm.so")
pytestmark = pytest.mark.skipif(not os.path.exists(LIB), reason="libqgemm.so not built")

M, K, N = 16, 256, 32
GIVEN = types.SimpleNamespace(device_index=-1, cuda_stream=7, name="given")   # -1: get_device() of a CPU tensor


@pytest.fixture
def recorded(monkeypatch):
    """(ops, events): (what, stream's name) of every allocation and launch."""
    from weight_only_quantized_w4a16_amd import ops
    events, current = [], ["current"]

    @contextlib.contextmanager
    def on(stream):
        before = current[0]
        current[0] = stream.name if stream is not None else before
        yield
        current[0] = before

    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: types.SimpleNamespace(name=current[0]))
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    for name in ("empty", "zeros"):
        real = getattr(torch, name)
        monkeypatch.setattr(torch, name, lambda *a, _real=real, _name=name, **k: (events.append((_name, current[0])), _real(*a, **k))[1])

    def launch(name):
        def f(*args, stream=None, **kw):
            given = stream or next((v for v in args if v is GIVEN), None)
            events.append((name, given.name if given else current[0]))
        return f
    for name in ("qgemm_w4a16", "qgemm_w4a16_epilogue", "qgemm_w8a8_fp8", "qgemm_w8a8_fp8_dynamic", "qgemm_w8a8_int8",
                 "qgemm_w8a8_int8_dynamic", "qgemm_w4a8_fp8", "qgemm_w4a16_grouped", "qgemm_w4a8_fp8_grouped",
                 "qgemm_w4a8_fp8_grouped_dynamic", "quant_act_per_token", "quant_act_per_token_int8", "pack_int4_g128",
                 "quant_weight_fp8_per_channel", "quant_weight_int8_per_channel", "dequant_int4_g128"):
        monkeypatch.setattr(ops, name, launch(name))
    for name in ("w4a16", "w8a8", "w8a8_int8", "w8a8_dynamic", "w4a16_grouped", "w4a8_grouped_dynamic"):
        monkeypatch.setattr(ops, name + "_workspace_bytes", lambda *a: 1024)
    return ops, events


bf = lambda *s: torch.ones(s, dtype=torch.bfloat16)
CALLS = {
    "W4A16Linear": lambda ops: ops.W4A16Linear(ops.Int4G128Weight(bf(1), bf(1), K, N))(bf(M, K), stream=GIVEN),
    "W4A16Linear with an epilogue": lambda ops: ops.W4A16Linear(ops.Int4G128Weight(bf(1), bf(1), K, N), bf(N), "silu")(
        bf(M, K), stream=GIVEN, residual=bf(M, N)),
    "W8A8Fp8Linear": lambda ops: ops.W8A8Fp8Linear(ops.Fp8Weight(bf(1), bf(1), K, N))(bf(M, K), stream=GIVEN),
    "W8A8Int8Linear": lambda ops: ops.W8A8Int8Linear(ops.Int8Weight(bf(1), bf(1), K, N))(bf(M, K), stream=GIVEN),
    "W4A8Linear": lambda ops: ops.W4A8Linear(ops.Int4G128Weight(bf(1), bf(1), K, N))(bf(M, K), stream=GIVEN),
    "grouped": lambda ops: ops.GroupedInt4Weight(bf(1), bf(1), 2, K, N)(bf(M, K), torch.ones(3, dtype=torch.int32), stream=GIVEN),
    "grouped w4a8": lambda ops: ops.GroupedInt4Weight(bf(1), bf(1), 2, K, N).w4a8(bf(M, K), bf(M), torch.ones(3, dtype=torch.int32),
                                                                                stream=GIVEN),
    "grouped w4a8 dynamic": lambda ops: ops.GroupedInt4Weight(bf(1), bf(1), 2, K, N).w4a8_dynamic(
        bf(M, K), torch.ones(3, dtype=torch.int32), stream=GIVEN),
    "quantize_activations": lambda ops: ops.quantize_activations(bf(M, K), stream=GIVEN),
    "quantize_activations_int8": lambda ops: ops.quantize_activations_int8(bf(M, K), stream=GIVEN),
    "pack": lambda ops: ops.Int4G128Weight.from_bf16(bf(K, N), stream=GIVEN).dequant(with_codes=True, stream=GIVEN),
    "pack grouped": lambda ops: ops.GroupedInt4Weight.from_bf16(bf(2, K, N), stream=GIVEN),
    "Fp8Weight": lambda ops: ops.Fp8Weight.from_bf16(bf(K, N), stream=GIVEN),
    "Int8Weight": lambda ops: ops.Int8Weight.from_bf16(bf(K, N), stream=GIVEN),
}


@pytest.mark.parametrize("what", CALLS)
def test_given_stream(recorded, what):
    ops, events = recorded
    CALLS[what](ops)
    assert any(n in ("empty", "zeros") for n, _ in events) and any(n not in ("empty", "zeros") for n, _ in events)
    assert {s for _, s in events} == {"given"}, events


def test_stream_of_another_device(recorded):
    ops, _ = recorded
    other = types.SimpleNamespace(device_index=3, cuda_stream=7, name="other")
    with pytest.raises(ValueError, match="another device"):
        ops.W4A16Linear(ops.Int4G128Weight(bf(1), bf(1), K, N))(bf(M, K), stream=other)


def test_outgrown_workspace_waits_for_the_calls_before(recorded, monkeypatch):
    """The last call may have used it on another stream than the one it came from: its memory goes back to that
    stream's pool only when the stream that replaces it, which follows that call, gets there."""
    ops, events = recorded
    told = []
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: told.append((t.numel(), s.name)))
    lin = ops.W4A16Linear(ops.Int4G128Weight(bf(1), bf(1), K, N))
    lin(bf(M, K))
    lin(bf(M, K), stream=GIVEN)
    assert not told
    monkeypatch.setattr(ops, "w4a16_workspace_bytes", lambda *a: 4096)
    lin(bf(M, K), stream=GIVEN)
    assert told == [(1024, "given")]


def test_workspace_of_a_capture(recorded, monkeypatch):
    """A capture's clearing runs in its replays only: a buffer that the capture brought is not kept for other calls.
    One that it found stays alive when later calls outgrow it."""
    ops, events = recorded
    capturing, need = [True], [1024]
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: capturing[0])
    monkeypatch.setattr(ops, "w4a16_workspace_bytes", lambda *a: need[0])
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: None)
    lin = ops.W4A16Linear(ops.Int4G128Weight(bf(1), bf(1), K, N))
    first, _ = lin.workspace(M)
    capturing[0] = False
    del events[:]
    held, _ = lin.workspace(M)
    assert held is not first and events == [("zeros", "current")]
    capturing[0] = True
    assert lin.workspace(M)[0] is held
    capturing[0], need[0] = False, 4096
    alive = weakref.ref(held)
    del held
    assert lin.workspace(M)[0].numel() == 4096 and alive() is not None
