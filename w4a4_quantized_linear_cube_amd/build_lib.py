"""Build libdq.so (HIP, gfx950) in-tree with hipcc, and _dqcall.so, the native
part of the Python binding, with g++ against torch's headers.

Each source compiles to its own object in `_build/` (in parallel), then one
link each makes the shared libraries next to this file.  Every call rebuilds.
_dqcall.so is left out, with a notice, where what it needs is not there
(libdq.so does not need it, and dq.py goes without).
"""
from __future__ import annotations

import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libdq.so")
SOURCES = ["api.cpp", "svd.cpp", "quant.hip", "gemm.hip", "noalloc.hip", "orbit.hip", "norm.hip", "rows.hip"]
CALL_LIB = os.path.join(HERE, "_dqcall.so")
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")

FLAGS = [
    "-O3", "-std=c++17", "-fPIC", "--offload-arch=gfx950",
    # packed fp32 VALU forms are kept out of every kernel
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    # no fused multiply-add contraction: the activation pass must round each step
    "-ffp-contract=off",
    "-Wall", "-Wno-unused-result",
    "-I", INCLUDE, "-I", CSRC,
]


def _torch_dir():
    spec = importlib.util.find_spec("torch")
    return os.path.dirname(spec.origin) if spec else None


def _call_lacks():
    """What _dqcall.so needs and this machine has not, or None."""
    t = _torch_dir()
    if shutil.which("g++") is None:
        return "g++"
    if t is None:
        return "torch"
    for name, path in (("torch's HIP headers", os.path.join(t, "include", "c10", "hip", "HIPStream.h")),
                       ("Python's headers", os.path.join(sysconfig.get_paths()["include"], "Python.h"))):
        if not os.path.isfile(path):
            return name
    return None


def _call_flags():
    t = os.path.join(_torch_dir(), "include")
    return ["-O2", "-std=c++17", "-fPIC", "-D__HIP_PLATFORM_AMD__", "-DUSE_ROCM", "-I", INCLUDE,
            "-I", sysconfig.get_paths()["include"], "-I", t, "-I", os.path.join(t, "torch", "csrc", "api", "include"),
            "-I", os.path.join(os.environ.get("ROCM_PATH", "/opt/rocm"), "include")]


def _start(cmd, verbose):
    if verbose:
        print(" ".join(cmd), flush=True)
    return subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)


def build(verbose: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    procs = []
    lacks = _call_lacks()
    call_obj = os.path.join(BUILD, "binding.o")
    call = None if lacks else _start(["g++", *_call_flags(), "-c", os.path.join(CSRC, "binding.cpp"), "-o", call_obj], verbose)
    objs = []
    for src in SOURCES:
        obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
        objs.append(obj)
        lang = ["-x", "hip"] if src.endswith(".hip") else []
        procs.append((src, _start([HIPCC, *FLAGS, *lang, "-c", os.path.join(CSRC, src), "-o", obj], verbose)))
    failed = []
    for src, p in procs:
        out, _ = p.communicate()
        out = "\n".join(l for l in out.splitlines() if "packed-fp32-ops" not in l and "unknown CPU feature" not in l
                        and l.strip() != "1 warning generated." and "is not a recognized feature" not in l)
        if out.strip() and (verbose or p.returncode):
            print(out, file=sys.stderr, flush=True)
        if p.returncode:
            failed.append(src)
    call_out = call.communicate()[0] if call else ""
    if failed:
        raise RuntimeError(f"hipcc failed for {failed}")
    tmp = LIB + ".tmp"
    cmd = [HIPCC, "-shared", "-fPIC", "--offload-arch=gfx950", *objs, "-o", tmp, "-lpthread"]
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.run(cmd, check=True)
    os.replace(tmp, LIB)
    # (one of an older build would call the new library by the old arguments)
    if os.path.exists(CALL_LIB):
        os.remove(CALL_LIB)
    if lacks:
        print(f"_dqcall.so is left out: {lacks} not found", file=sys.stderr, flush=True)
        return LIB
    tmp = CALL_LIB + ".tmp"
    if call.returncode == 0:
        call = _start(["g++", "-shared", call_obj, "-o", tmp, "-L", HERE, "-ldq", "-Wl,-rpath,$ORIGIN", "-L",
                       os.path.join(_torch_dir(), "lib"), "-lc10", "-lc10_hip", "-ltorch_cpu", "-ltorch_python"], verbose)
        call_out = call.communicate()[0]
    if call.returncode:
        print(call_out, file=sys.stderr, flush=True)
        raise RuntimeError("g++ failed for _dqcall.so (libdq.so is built)")
    os.replace(tmp, CALL_LIB)
    return LIB


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
