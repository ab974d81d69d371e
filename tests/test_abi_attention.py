"""The operators between the qkv product and the o product reject invalid arguments on the host, before anything is
launched.  Runs without a GPU: every call fails validation (or has nothing to do), so the pointers are never dereferenced."""
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
    assert set(changed) <= set(defaults), changed
    return getattr(ops._lib, name)(*dict(defaults, **changed).values(), None)


ROPE = dict(qkv=FAKE, wq=FAKE, wk=FAKE, eps=1e-6, positions=FAKE, freq=FAKE, rot=128, inter=0, T=4, Hq=8, Hkv=2, D=128, q=FAKE,
            k=FAKE)
APPEND = dict(qkv=FAKE, wq=FAKE, wk=FAKE, eps=1e-6, freq=FAKE, rot=128, inter=0, offsets=FAKE, len=FAKE, table=FAKE, T=4, B=2,
              width=8, Hq=8, Hkv=2, D=128, k=FAKE, v=FAKE, ks=FAKE, vs=FAKE, pages=20, page=16, q=FAKE)
ATTEND = dict(q=FAKE, k=FAKE, v=FAKE, ks=FAKE, vs=FAKE, pages=20, page=16, offsets=FAKE, len=FAKE, table=FAKE, T=4, B=2, width=8,
              Hq=8, Hkv=2, D=128, scale=0.1, window=0, sinks=0, shared=0, max_q=0, out=FAKE, lse=FAKE, ws=FAKE, bytes=1 << 40)
HEADS = [dict(T=-1), dict(T=1 << 22), dict(Hq=0), dict(Hkv=0), dict(Hq=9), dict(Hq=1, Hkv=2), dict(Hq=1026, Hkv=2), dict(D=32),
         dict(D=96), dict(D=256), dict(T=1 << 20, Hq=256)]
LISTS = [dict(B=-1), dict(B=(1 << 14) + 1), dict(width=0), dict(width=-1), dict(width=1 << 27), dict(page=0), dict(page=8),
         dict(page=17), dict(page=512), dict(page=-16), dict(pages=0), dict(pages=-1)]
FREE = ("eps", "rot", "inter", "T", "B", "width", "Hq", "Hkv", "D", "pages", "page", "scale", "window", "sinks", "shared", "max_q", "bytes")


@pytest.mark.parametrize("name,base", [("qk_norm_rope", ROPE), ("kv_append", APPEND)])
def test_rope_refusals(ops, name, base):
    for changed in HEADS + [dict(rot=-16), dict(rot=8), dict(rot=144)] + \
            [dict(eps=e) for e in (0.0, -1.0, 1e-39, float("inf"), float("nan"))] + (LISTS if base is APPEND else []):
        assert call(ops, name, base, **changed) == QG_ERR_SHAPE, changed
    for p in set(base) - set(FREE):
        if p not in ("wq", "wk"):
            assert call(ops, name, base, **{p: None}) == QG_ERR_NULL, p
        assert call(ops, name, base, **{p: FAKE + 2}) == QG_ERR_ALIGN, p
    assert call(ops, name, base, T=0, qkv=None) == QG_OK
    assert call(ops, name, base, wq=None, wk=None, eps=0.0, q=None) == QG_ERR_NULL      # no norm: eps is not read


def test_append_of_no_sequences(ops):
    assert call(ops, "kv_append", APPEND, B=0, qkv=None) == QG_OK


def test_attention_refusals(ops):
    for changed in HEADS + LISTS + [dict(scale=float("nan")), dict(scale=float("inf")), dict(window=-1),
                                    dict(window=(1 << 30) + 1), dict(sinks=-1), dict(shared=-16), dict(shared=8),
                                    dict(shared=144), dict(max_q=-1)]:
        assert call(ops, "paged_attention", ATTEND, **changed) == QG_ERR_SHAPE, changed
    for p in set(ATTEND) - set(FREE):
        if p not in ("lse", "ws"):
            assert call(ops, "paged_attention", ATTEND, **{p: None}) == QG_ERR_NULL, p
        if p != "ws":
            assert call(ops, "paged_attention", ATTEND, **{p: FAKE + 2}) == QG_ERR_ALIGN, p
    assert call(ops, "paged_attention", ATTEND, T=0, q=None) == QG_OK
    assert call(ops, "paged_attention", ATTEND, B=0, q=None) == QG_OK


def test_attention_workspace(ops):
    big = dict(ATTEND, width=4096)
    need = ops.paged_attention_workspace_bytes(4, 2, 4096, 8, 2, 128, 16)
    assert need > 65536
    assert call(ops, "paged_attention", big, ws=None) == QG_ERR_NULL
    assert call(ops, "paged_attention", big, bytes=need - 1) == QG_ERR_WORKSPACE
    assert call(ops, "paged_attention", big, ws=FAKE + 8) == QG_ERR_ALIGN


def test_workspace_query_of_bad_sizes(ops):
    ok = dict(T=4, B=2, width=4096, Hq=8, Hkv=2, D=128, page=16, shared=0, max_q=0)
    assert ops.paged_attention_workspace_bytes(*ok.values()) > 0
    for changed in HEADS + LISTS[:10] + [dict(shared=-16), dict(shared=8), dict(max_q=-1), dict(width=2 ** 62), dict(B=2 ** 62),
                                         dict(T=2 ** 62), dict(Hq=2 ** 62), dict(page=2 ** 62), dict(page=16 - 2 ** 32)]:
        assert ops.paged_attention_workspace_bytes(*dict(ok, **changed).values()) == 0, changed
    assert ops.paged_attention_workspace_bytes(*dict(ok, T=0).values()) == 0
    assert ops.paged_attention_workspace_bytes(*dict(ok, B=0).values()) == 0
