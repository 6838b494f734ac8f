"""Build libomm.so (the C-ABI library with the gfx950 kernels) and _native.so (the
Python binding of the decode-side operators) in the package dir.

    python -m onnx_matmul_family_amd.build          # or build() from Python

Every source is compiled with hipcc for gfx950 only.  Packed-fp32 VALU forms
are disabled (-packed-fp32-ops) and the QLinearMatMul requantisation file is
built without floating-point contraction, so its fp32 steps stay separately
rounded.
"""
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libomm.so")
NATIVE = os.path.join(HERE, "_native.so")
BUILD = os.path.join(HERE, "_build")

SOURCES = ["api.cpp", "dense16.hip", "dense_f32.hip", "dense_f64.hip", "qlinear.hip", "grouped.hip",
           "moe.hip", "lora.hip", "lora_rows.hip", "token_logprobs.hip", "int8.hip",
           "moe_balance.hip", "orthogonal.hip"]
COMMON = ["--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC", "-Wall",
          "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
          "-I", os.path.join(HERE, "..", "include")]
PER_FILE = {"qlinear.hip": ["-ffp-contract=off"]}


def hipcc():
    for c in (os.environ.get("HIPCC"), "/opt/rocm/bin/hipcc", shutil.which("hipcc")):
        if c and os.path.exists(c):
            return c
    raise RuntimeError("hipcc not found")


def _compile(src, verbose):
    obj = os.path.join(BUILD, src + ".o")
    lang = ["-x", "hip"] if src.endswith(".cpp") else []
    cmd = [hipcc()] + COMMON + PER_FILE.get(src, []) + lang + ["-c", os.path.join(CSRC, src), "-o", obj]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("compile failed: %s\n%s\n%s" % (src, r.stdout, r.stderr))
    return obj


def _build_native(verbose):
    """csrc/binding.cpp against the installed torch (host code only)."""
    import torch
    base = os.path.dirname(torch.__file__)
    rocm = os.path.dirname(os.path.dirname(os.path.realpath(hipcc())))
    lib = os.path.join(base, "lib")
    cmd = [hipcc(), "-no-hip-rt", "-x", "c++", "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall", "-D__HIP_PLATFORM_AMD__=1",
           "-DUSE_ROCM", "-D_GLIBCXX_USE_CXX11_ABI=%d" % torch._C._GLIBCXX_USE_CXX11_ABI,
           "-I", os.path.join(HERE, "..", "include"), "-isystem", os.path.join(base, "include"),
           "-isystem", os.path.join(base, "include", "torch", "csrc", "api", "include"),
           "-isystem", sysconfig.get_paths()["include"], "-isystem", os.path.join(rocm, "include"),
           os.path.join(CSRC, "binding.cpp"), "-x", "none", "-o", NATIVE + ".tmp", "-L", lib, "-Wl,-rpath," + lib,
           "-ltorch_python", "-ltorch_cpu", "-ltorch", "-lc10", "-lc10_hip"]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("compile failed: binding.cpp\n%s\n%s" % (r.stdout, r.stderr))
    os.replace(NATIVE + ".tmp", NATIVE)


def build(verbose=False, jobs=None):
    """libomm.so, then _native.so, which only a Python with torch needs: without torch the
    library is all there is to build."""
    os.makedirs(BUILD, exist_ok=True)
    jobs = jobs or min(len(SOURCES), max(1, (os.cpu_count() or 4)))
    with ThreadPoolExecutor(jobs) as ex:
        objs = list(ex.map(lambda s: _compile(s, verbose), SOURCES))
    tmp = LIB + ".tmp"
    cmd = [hipcc(), "--offload-arch=gfx950", "-shared", "-fPIC", "-o", tmp] + objs
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.check_call(cmd)
    os.replace(tmp, LIB)
    if importlib.util.find_spec("torch") is None:
        print("torch is not installed: _native.so is not built", file=sys.stderr)
    else:
        _build_native(verbose)
    return LIB


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
