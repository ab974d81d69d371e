"""The compiled call marshalling belongs to one interpreter and one torch; without
it the library's products work as before and the calls that go through it say
what is missing."""
import os
import subprocess
import sys
import sysconfig

import pytest

from conftest import ROOT

LIB = os.path.join(ROOT, "weight_only_quantized_w4a16_amd", "libqgemm.so")
built = pytest.mark.skipif(not os.path.exists(LIB), reason="libqgemm.so not built")

WITHOUT = {
    "absent": "None",
    "of another torch": "types.SimpleNamespace(torch_version='0.1', swiglu=None)",
    "of an unknown torch": "types.SimpleNamespace(swiglu=None)",
}


@built
@pytest.mark.parametrize("case", WITHOUT)
def test_products_without_the_marshalling(case):
    code = f"""
import sys, types
sys.modules["weight_only_quantized_w4a16_amd._calls"] = {WITHOUT[case]}
from weight_only_quantized_w4a16_amd import ops
assert ops.packed_bytes(128, 16) == 1024
assert ops.w4a16_kernel_for(1, 4096, 4096)
assert ops.moe_dispatch_workspace_bytes(65536, 8, 128) > 0
assert ops.qgemm_w4a16 and ops.W4A16Linear
for call in (lambda: ops.swiglu(None, 2, 64, None), lambda: ops.rms_norm(None, None, None, 1e-5, 2, 64, None, None),
             lambda: ops.moe_combine(None, None, None, None, 1, 1, 8, None)):
    try:
        call()
    except ImportError as e:
        assert "weight_only_quantized_w4a16_amd.build" in str(e), e
    else:
        raise SystemExit("a call without its marshalling did not raise")
"""
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


@built
def test_the_marshalling_names_its_torch():
    import torch
    from weight_only_quantized_w4a16_amd import _calls
    assert _calls.torch_version == torch.__version__
    assert _calls.__file__.endswith(sysconfig.get_config_var("EXT_SUFFIX"))


def test_the_library_is_built_without_the_marshalling(monkeypatch, tmp_path):
    """A machine without a C++ compiler or torch's headers still gets libqgemm.so, and the reason."""
    from weight_only_quantized_w4a16_amd import build

    def fail():
        raise RuntimeError("no headers")

    def link(cmd, **kw):
        open(cmd[cmd.index("-o") + 1], "w").close()
        return subprocess.CompletedProcess(cmd, 0, "", "")
    monkeypatch.setattr(build, "_build_calls", fail)
    monkeypatch.setattr(build, "_compile", lambda src: (src, ""))
    monkeypatch.setattr(build, "LIB", str(tmp_path / "libqgemm.so"))
    monkeypatch.setattr(build.subprocess, "run", link)
    with pytest.raises(RuntimeError, match="no headers"):
        build.build(verbose=False)
    assert os.path.exists(tmp_path / "libqgemm.so")
