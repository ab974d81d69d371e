"""perf/operators.py: the plain forms agree with the definitions in 64 bits on small
cases, and the listed and drawn cases are sizes that the library accepts.  CPU only."""
import random

import pytest
import torch

from perf import operators

SMALL = [dict(op="norm", M=5, K=64, out=o, residual=r) for o in ("bf16", "e4m3", "int8") for r in (True, False)] + \
        [dict(op="swiglu", M=5, I=64, out=o) for o in ("bf16", "e4m3", "int8")] + \
        [dict(op="dispatch", B=9, k=3, E=8, K=16, out=o, dropped=0.2) for o in ("bf16", "e4m3")] + \
        [dict(op="combine", B=9, k=3, E=8, K=16, residual=r, dropped=0.2) for r in (True, False)] + \
        [dict(op="combine_backward", B=9, k=3, E=8, K=16, dropped=0.2)] + \
        [dict(op="linear", M=5, K=256, N=32, bias=True, act=a, residual=True)
         for a in ("none", "relu", "gelu", "gelu_tanh", "silu")]


@pytest.mark.parametrize("case", SMALL, ids=str)
def test_plain_forms(case, monkeypatch):
    monkeypatch.setattr(operators, "DEV", "cpu")
    got, want = operators.run(operators.prepare(case, 3)), operators.exact(case, 3)
    assert set(got) == set(want)
    for name, x in got.items():
        y = want[name].double()
        # half a step of the output's type at every value: 2^-4 e4m3, 2^-8 bf16; fp32 sums of up to 256 terms
        step = {torch.float8_e4m3fn: 2.0 ** -4, torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -16, torch.int32: 0.0}[x.dtype]
        tiny = 2.0 ** -10 if x.dtype == torch.float8_e4m3fn else 1e-6
        assert ((x.double() - y).abs() <= step * (1 + 2.0 ** -7) * y.abs() + (tiny if step else 0)).all(), name


def test_cases():
    listed = operators.listed()
    assert 4 <= len(listed) <= 12 and len({c["name"] for c in listed}) == len(listed)
    rng = random.Random(1)
    top = max(max(operators.work(c)["bytes"], operators.work(c)["flops"] / 50) for c in listed)
    for c in listed + [operators.draw(rng) for _ in range(200)]:
        w = operators.work(c)
        assert 0 < w["bytes"] and max(w["bytes"], w["flops"] / 50) <= 1.05 * top
        if c["op"] == "linear":
            assert c["K"] % 128 == 0 and c["N"] % 16 == 0
        else:
            assert c.get("K", c.get("I")) % 8 == 0
