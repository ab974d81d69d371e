"""The launches of paged_attention at the ends of the sizes that it accepts, recorded by a host build of its launcher and
argument checks against a runtime that launches nothing (tests/asan/attention_launches.cpp).  No GPU is needed."""
import os
import subprocess

import pytest

from conftest import ROOT

ROCM = "/opt/rocm"
HIPCC = os.environ.get("HIPCC", os.path.join(ROCM, "bin", "hipcc"))


@pytest.mark.skipif(not os.path.exists(HIPCC), reason="needs hipcc")
def test_every_launch_fits_its_grid(tmp_path):
    csrc = os.path.join(ROOT, "weight_only_quantized_w4a16_amd", "csrc")
    include = ["-std=c++17", "-O1", "-fPIE", "-I", csrc]
    for_host = ["g++", *include, "-D__HIP_PLATFORM_AMD__", "-I", os.path.join(ROCM, "include")]
    for_launches = [HIPCC, *include, "--offload-arch=gfx950", "--offload-host-only", "-fuse-cuid=none", "-Wno-unused-command-line-argument"]
    objects = []
    for command, src in ((for_launches, os.path.join(csrc, "attention.hip")), (for_host, os.path.join(csrc, "abi_attention.cpp")),
                         (for_host, os.path.join(ROOT, "tests", "asan", "attention_launches.cpp"))):
        obj = str(tmp_path / (os.path.basename(src) + ".o"))
        r = subprocess.run([*command, "-c", src, "-o", obj], capture_output=True, text=True)
        assert r.returncode == 0, r.stderr[-4000:]
        objects.append(obj)
    exe = str(tmp_path / "attention_launches")
    r = subprocess.run(["g++", *objects, "-o", exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-4000:]
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and "attention launches ok" in r.stdout, (r.stdout + r.stderr)[-4000:]
