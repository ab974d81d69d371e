"""perf/more_operators.py: the plain forms agree with the definitions in 64 bits on small cases, and the listed and drawn
cases are sizes that the library accepts.  CPU only."""
import random

import pytest
import torch

from perf import more_operators as cases

ROPE = dict(Hq=4, Hkv=2, D=64)
SMALL = [dict(ROPE, op="norm_rope", T=5, norm=n, rot=r, inter=i) for n in (True, False) for r in (64, 32) for i in (True, False)] + \
        [dict(ROPE, op="append", B=3, n=5, ragged=True, kv=40, page=16, fmt=f, norm=True, rot=64, inter=False) for f in ("bf16", "e4m3")] + \
        [dict(ROPE, op="attend", B=3, n=n, ragged=True, kv=70, page=16, fmt=f, window=w, sinks=s, lse=True)
         for f in ("bf16", "e4m3") for n in (1, 9) for w, s in ((0, 0), (8, 2), (1, 0), (100, 4))] + \
        [dict(ROPE, op="shared", B=3, n=n, ragged=True, prefix=32, kv=60, page=16, fmt=f, lse=True)
         for f in ("bf16", "e4m3") for n in (1, 3)]


@pytest.mark.parametrize("case", SMALL, ids=str)
def test_plain_forms(case, monkeypatch):
    monkeypatch.setattr(cases, "DEV", "cpu")
    got, want = cases.run(cases.prepare(case, 3)), cases.exact(case, 3)
    assert set(got) == set(want)
    for name, x in got.items():
        y = want[name].double()
        # half a step of the output's type at every value (2^-4 e4m3, 2^-8 bf16) and fp32 work of values up to some 10
        step = {torch.float8_e4m3fn: 2.0 ** -4, torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -20}[x.dtype]
        tiny = 2.0 ** -9 if x.dtype == torch.float8_e4m3fn else 2e-5
        assert ((x.double() - y).abs() <= step * (1 + 2.0 ** -7) * y.abs() + tiny).all(), name


def test_cases():
    listed = cases.listed()
    assert 4 <= len(listed) <= 12 and len({c["name"] for c in listed}) == len(listed)
    rng = random.Random(1)
    cost = lambda c: max(cases.work(c)["bytes"], cases.work(c)["flops"] / 50)
    top = max(cost(c) for c in listed)
    for c in listed + [cases.draw(rng) for _ in range(200)]:
        assert 0 < cost(c) <= top
        assert c["Hq"] % c["Hkv"] == 0 and c["D"] in (64, 128) and c.get("rot", 0) % 16 == 0
        assert c.get("page", 16) in (16, 32, 64, 128, 256) and c.get("prefix", 0) % c.get("page", 16) == 0
