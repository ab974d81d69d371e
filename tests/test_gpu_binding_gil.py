"""The compiled marshalling lets other Python threads run during a call.

A launch waits while the device's queue is full, and what empties the queue may be
waiting for another Python thread.  Here `swiglu` stands for any call: its address
is replaced by libc's poll(no descriptors, none, 300 ms), which does nothing but
wait and returns 0.
"""
import ctypes
import threading
import time

import pytest
import torch

from gpu_helpers import announce

pytestmark = pytest.mark.gpu


def test_other_threads_run_during_a_call():
    from weight_only_quantized_w4a16_amd import ops
    announce("binding releases the interpreter lock")
    y = torch.zeros((2, 64), dtype=torch.bfloat16, device="cuda:0")   # gives the call its device
    address = lambda f: ctypes.cast(f, ctypes.c_void_p).value
    spans = []

    def call():
        t = time.monotonic()
        ops.swiglu(None, 0, 300, y)                                   # poll(NULL, 0, 300)
        spans.append((t, time.monotonic()))

    ticks = []
    ops._calls.bind("swiglu", address(ctypes.CDLL(None).poll))
    try:
        thread = threading.Thread(target=call)
        thread.start()
        while thread.is_alive():
            ticks.append(time.monotonic())
            time.sleep(0.005)
        thread.join()
    finally:
        ops._calls.bind("swiglu", address(ops._lib.swiglu))
    (t0, t1), = spans
    assert t1 - t0 > 0.25
    during = sum(t0 + 0.01 < t < t1 - 0.01 for t in ticks)
    assert during >= 5, f"{during} ticks of another thread in {t1 - t0:.2f} s"
