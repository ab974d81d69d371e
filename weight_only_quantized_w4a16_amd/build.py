"""Build libqgemm.so in-tree with hipcc for gfx950, and the _calls extension, the
binding's call marshalling (host code against the installed torch's headers; its
file name carries the interpreter's ABI, the module the torch it was built with).
The library is there also when the extension cannot be built; the reason is raised
after it.

    python -m weight_only_quantized_w4a16_amd.build

Every call compiles from source (no staleness check): the object files go to
csrc/_build/, the libraries to the package directory.
"""
import concurrent.futures
import importlib.util
import os
import runpy
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(CSRC, "_build")
LIB = os.path.join(PKG, "libqgemm.so")
CALLS = os.path.join(PKG, "_calls" + sysconfig.get_config_var("EXT_SUFFIX"))
SOURCES = ["abi.cpp", "abi_block.cpp", "w4a16.hip", "fp8.hip", "w4a8.hip", "norm.hip", "moe.hip",
           "abi_attention.cpp", "rope.hip", "attention.hip"]
ARCH = "gfx950"

HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
CXX = os.environ.get("CXX", "g++")
ROCM = os.environ.get("ROCM_PATH", "/opt/rocm")

COMMON_FLAGS = [
    "-O3", "-std=c++17", "-fPIC", f"--offload-arch={ARCH}",
    "-Wall", "-Wno-unused-command-line-argument",
    # an inline-asm warning (e.g. a clobbered reserved register) fails the build
    "-Werror=inline-asm",
    # keep the compiler from forming packed-fp32 VALU instructions
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-I", os.path.join(ROOT, "include"),
]


def _compile(src):
    obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
    cmd = [HIPCC, *COMMON_FLAGS, "-c", os.path.join(CSRC, src), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"hipcc failed for {src}:\n{' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    warn = "\n".join(l for l in r.stderr.splitlines() if "packed-fp32-ops" not in l and l.strip())
    return obj, warn


def _build_calls():
    torch = importlib.util.find_spec("torch").submodule_search_locations[0]
    lib = os.path.join(torch, "lib")
    version = runpy.run_path(os.path.join(torch, "version.py"))["__version__"]
    tmp = CALLS + ".tmp"
    cmd = [CXX, "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall", "-D__HIP_PLATFORM_AMD__", "-DUSE_ROCM",
           f'-DQG_TORCH_VERSION="{version}"',
           "-I", os.path.join(torch, "include"), "-I", os.path.join(ROCM, "include"),
           "-I", sysconfig.get_paths()["include"], os.path.join(CSRC, "calls.cpp"),
           "-L", lib, "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_hip",
           "-L", os.path.join(ROCM, "lib"), "-lamdhip64", "-Wl,-rpath," + lib, "-o", tmp]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{CXX} failed for calls.cpp:\n{' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, CALLS)


def build(verbose=True):
    os.makedirs(BUILD, exist_ok=True)
    with concurrent.futures.ThreadPoolExecutor(len(SOURCES) + 1) as ex:
        calls = ex.submit(_build_calls)
        results = list(ex.map(_compile, SOURCES))
    objs = [o for o, _ in results]
    if verbose:
        for (_, w), src in zip(results, SOURCES):
            if w:
                print(f"[{src}] {w}", file=sys.stderr)
    tmp = LIB + ".tmp"
    cmd = [HIPCC, f"--offload-arch={ARCH}", "-shared", "-fPIC", *objs, "-o", tmp]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    if verbose:
        print(f"built {LIB}")
    calls.result()
    if verbose:
        print(f"built {CALLS}")
    return LIB


if __name__ == "__main__":
    build()
