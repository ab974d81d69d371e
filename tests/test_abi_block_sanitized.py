"""abi_block.cpp built for the host with AddressSanitizer and
UndefinedBehaviorSanitizer against stub launchers (tests/asan/block_*.cpp):
extreme sizes overflow nothing, and refused calls launch nothing.  Host code
only; no GPU is needed."""
import os
import shutil
import subprocess

import pytest

from conftest import ROOT

ROCM = "/opt/rocm"


@pytest.mark.skipif(shutil.which("g++") is None or not os.path.isdir(os.path.join(ROCM, "include", "hip")),
                    reason="needs g++ and the HIP headers")
def test_abi_block_under_host_sanitizers(tmp_path):
    exe = tmp_path / "abi_block_driver"
    csrc = os.path.join(ROOT, "weight_only_quantized_w4a16_amd", "csrc")
    asan = os.path.join(ROOT, "tests", "asan")
    cmd = ["g++", "-std=c++17", "-g", "-O1", "-fsanitize=address,undefined", "-fno-omit-frame-pointer",
           "-fno-sanitize-recover=undefined", "-D__HIP_PLATFORM_AMD__", "-I", os.path.join(ROCM, "include"), "-I", csrc,
           os.path.join(csrc, "abi_block.cpp"), os.path.join(asan, "block_stubs.cpp"),
           os.path.join(asan, "block_driver.cpp"),
           "-L", os.path.join(ROCM, "lib"), "-lamdhip64", "-Wl,-rpath," + os.path.join(ROCM, "lib"), "-o", str(exe)]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-4000:]
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0", UBSAN_OPTIONS="print_stacktrace=1")
    r = subprocess.run([str(exe)], capture_output=True, text=True, env=env, timeout=120)
    assert r.returncode == 0, (r.stdout + r.stderr)[-4000:]
    assert "abi block driver ok" in r.stdout
