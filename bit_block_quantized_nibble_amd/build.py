"""Compile libqbn.so (the HIP kernels and the C ABI) for gfx950 with hipcc.

Each .hip source under csrc/ is compiled to an object in _build/ (in
parallel), then linked into bit_block_quantized_nibble_amd/libqbn.so, next
to this file, so that the built library travels with the source tree. Next to
it, _kvcall.so: the Python module that makes the calls of the paged cache, the
rotation by positions and the experts' layer (host code, csrc/*.cpp, built with g++
against Python's and torch's headers and linked to libqbn.so). Where that one
cannot be built, the library is all the same, and everything but those Python
calls runs; the error comes last.

    python -m bit_block_quantized_nibble_amd.build
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import importlib.util
import os
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libqbn.so")
CALLS = os.path.join(HERE, "_kvcall.so")
INCLUDE = os.path.join(os.path.dirname(HERE), "include")

HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
ARCH = "gfx950"

# -packed-fp32-ops: keep the compiler from forming packed binary32 ops.
CFLAGS = [
    "-O3", "-std=c++17", "-fPIC", f"--offload-arch={ARCH}", "-fno-gpu-rdc", "-fvisibility=hidden",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wno-unused-command-line-argument", f"-I{INCLUDE}",
]


def _compile(src: str) -> str:
    obj = os.path.join(BUILD, os.path.basename(src) + ".o")
    cmd = [HIPCC, *CFLAGS, "-c", src, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("hipcc failed for %s:\n%s\n%s" % (src, r.stdout, r.stderr))
    return obj


def _compile_call(src: str) -> str:
    torch = os.path.dirname(importlib.util.find_spec("torch").origin)
    obj = os.path.join(BUILD, os.path.basename(src) + ".o")
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", "-I" + sysconfig.get_path("include"),
           "-I" + os.path.join(torch, "include"), "-I" + os.path.join(torch, "include", "torch", "csrc", "api", "include"),
           "-c", src, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("g++ failed for %s:\n%s\n%s" % (src, r.stdout, r.stderr))
    return obj


def _link_calls(objs: list) -> None:
    torch = os.path.dirname(importlib.util.find_spec("torch").origin)
    tmp = CALLS + ".tmp%d" % os.getpid()
    cmd = ["g++", "-shared", "-o", tmp, *objs, "-L" + HERE, "-l:libqbn.so", "-Wl,-rpath,$ORIGIN",
           "-L" + os.path.join(torch, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("linking _kvcall.so failed:\n%s\n%s" % (r.stdout, r.stderr))
    os.replace(tmp, CALLS)


def build(verbose: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    srcs = sorted(glob.glob(os.path.join(CSRC, "*.hip")))
    jobs = min(len(srcs), max(1, min(8, os.cpu_count() or 1)))
    with cf.ThreadPoolExecutor(jobs) as ex:
        calls = [ex.submit(_compile_call, src) for src in sorted(glob.glob(os.path.join(CSRC, "*.cpp")))]
        objs = list(ex.map(_compile, srcs))
    tmp = LIB + ".tmp%d" % os.getpid()
    cmd = [HIPCC, "-shared", "-fPIC", f"--offload-arch={ARCH}", "-fno-gpu-rdc", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("hipcc link failed:\n%s\n%s" % (r.stdout, r.stderr))
    os.replace(tmp, LIB)
    try:
        _link_calls([c.result() for c in calls])
    except Exception as e:
        if os.path.exists(CALLS):  # of another build: it may not fit this library
            os.remove(CALLS)
        raise RuntimeError("%s is built, but not %s, which makes the Python calls of the paged "
                           "cache, the rotation and the experts' layer" % (LIB, CALLS)) from e
    if verbose:
        print("built", LIB, CALLS)
    return LIB


if __name__ == "__main__":
    build(verbose=True)
    sys.exit(0)
