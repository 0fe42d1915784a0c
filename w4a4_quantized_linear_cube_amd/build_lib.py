"""Build libdq.so (HIP, gfx950) in-tree with hipcc, and _dqcall.so, the native
part of the Python binding, with g++ against torch's headers.

Each source compiles to its own object in `_build/` (in parallel), then one
link each makes the shared libraries next to this file.  Every call rebuilds.
"""
from __future__ import annotations

import os
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


def _torch_dir() -> str:
    import importlib.util
    return os.path.dirname(importlib.util.find_spec("torch").origin)


def _call_flags():
    t = os.path.join(_torch_dir(), "include")
    return ["-O2", "-std=c++17", "-fPIC", "-D__HIP_PLATFORM_AMD__", "-DUSE_ROCM", "-I", INCLUDE,
            "-I", sysconfig.get_paths()["include"], "-I", t, "-I", os.path.join(t, "torch", "csrc", "api", "include"),
            "-I", os.path.join(os.environ.get("ROCM_PATH", "/opt/rocm"), "include")]


def build(verbose: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    procs = []
    call_obj = os.path.join(BUILD, "binding.o")
    procs.append(("binding.cpp", subprocess.Popen(["g++", *_call_flags(), "-c", os.path.join(CSRC, "binding.cpp"), "-o", call_obj],
                                                  stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)))
    objs = []
    for src in SOURCES:
        obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
        objs.append(obj)
        lang = ["-x", "hip"] if src.endswith(".hip") else []
        cmd = [HIPCC, *FLAGS, *lang, "-c", os.path.join(CSRC, src), "-o", obj]
        if verbose:
            print(" ".join(cmd), flush=True)
        procs.append((src, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)))
    failed = []
    for src, p in procs:
        out, _ = p.communicate()
        out = "\n".join(l for l in out.splitlines() if "packed-fp32-ops" not in l and "unknown CPU feature" not in l
                        and l.strip() != "1 warning generated." and "is not a recognized feature" not in l)
        if out.strip() and (verbose or p.returncode):
            print(out, file=sys.stderr, flush=True)
        if p.returncode:
            failed.append(src)
    if failed:
        raise RuntimeError(f"hipcc failed for {failed}")
    tmp = LIB + ".tmp"
    cmd = [HIPCC, "-shared", "-fPIC", "--offload-arch=gfx950", *objs, "-o", tmp, "-lpthread"]
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.run(cmd, check=True)
    os.replace(tmp, LIB)
    tmp = CALL_LIB + ".tmp"
    lib = os.path.join(_torch_dir(), "lib")
    subprocess.run(["g++", "-shared", call_obj, "-o", tmp, "-L", HERE, "-ldq", "-Wl,-rpath,$ORIGIN", "-L", lib, "-lc10", "-lc10_hip",
                    "-ltorch_cpu", "-ltorch_python"], check=True)
    os.replace(tmp, CALL_LIB)
    return LIB


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
