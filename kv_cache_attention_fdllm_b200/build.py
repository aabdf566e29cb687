"""Builds libfdllm.so in-tree from csrc/*.cu for sm_100a with nvcc, and the binding's
short way to it (_fast, csrc/fast_call.cpp) with the host compiler against torch's headers.

Usage: python kv_cache_attention_fdllm_b200/build.py [--force] [-v] [--ptxas]
(run it by path: importing the package itself requires the built library)
Objects go to <repo>/_build/ (not committed); the shared library is written
next to this file so that it travels with the source tree.
"""
from __future__ import annotations

import argparse
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libfdllm.so")
FAST = os.path.join(PKG, "_fast.so")
FAST_FOR = os.path.join(BUILD, "fast_for.txt")  # what FAST was built for

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall",
         "--expt-relaxed-constexpr", "-I", INCLUDE, "-I", CSRC]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", shutil.which("nvcc")):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libfdllm.so")


def _sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def _headers_mtime():
    hs = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cuh", ".h"))]
    hs += [os.path.join(INCLUDE, f) for f in os.listdir(INCLUDE) if f.endswith(".h")]
    return max((os.path.getmtime(h) for h in hs), default=0.0)


def _torch() -> str:
    # found, not imported: importing torch takes longer than the compilation it is for
    return os.path.dirname(importlib.util.find_spec("torch").origin)


def _fast_made_for() -> str:
    """What a _fast.so belongs to: the torch it is compiled against and the interpreter."""
    with open(os.path.join(_torch(), "version.py")) as f:
        return f"{_torch()}\n{f.read()}\n{sys.version}\n"


def _fast_stale() -> bool:
    src = os.path.join(CSRC, "fast_call.cpp")
    if not os.path.exists(FAST) or not os.path.exists(FAST_FOR) or \
            os.path.getmtime(FAST) < max(os.path.getmtime(src), _headers_mtime()):
        return True
    with open(FAST_FOR) as f:
        return f.read() != _fast_made_for()


def _fast_command(cc) -> list:
    torch = _torch()
    inc = os.path.join(torch, "include")
    cuda = os.path.join(os.path.dirname(os.path.dirname(cc)), "include")
    libs = os.path.join(torch, "lib")
    return ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall", os.path.join(CSRC, "fast_call.cpp"),
            "-o", FAST, "-I", INCLUDE, "-isystem", inc, "-isystem", os.path.join(inc, "torch", "csrc", "api", "include"),
            "-isystem", sysconfig.get_paths()["include"], "-isystem", cuda, "-L", PKG, "-l:libfdllm.so",
            "-L", libs, "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda", "-Wl,-rpath,$ORIGIN"]


def build(force: bool = False, verbose: bool = False, ptxas_verbose: bool = False) -> str:
    """Compile every kernel source for sm_100a, link libfdllm.so and _fast.so; returns the
    former's path."""
    os.makedirs(BUILD, exist_ok=True)
    cc = nvcc()
    hdr = _headers_mtime()
    srcs = _sources()
    objs = []
    jobs = []
    for s in srcs:
        o = os.path.join(BUILD, os.path.basename(s)[:-3] + ".o")
        objs.append(o)
        stale = force or not os.path.exists(o) or os.path.getmtime(o) < max(os.path.getmtime(s), hdr)
        if stale:
            cmd = [cc] + ARCH + FLAGS + (["-Xptxas", "-v"] if ptxas_verbose else []) + ["-c", s, "-o", o]
            jobs.append(cmd)

    def run(cmd):
        if verbose:
            print(" ".join(cmd), flush=True)
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"failed: {' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
        if verbose or ptxas_verbose:
            sys.stdout.write(r.stdout + r.stderr)
        return r

    with ThreadPoolExecutor(max(1, min(8, os.cpu_count() or 1))) as ex:
        list(ex.map(run, jobs))
    if jobs or force or not os.path.exists(LIB) or \
            os.path.getmtime(LIB) < max(os.path.getmtime(o) for o in objs):
        cmd = [cc] + ARCH + ["-shared", "-o", LIB] + objs + ["-lcudart_static", "-ldl", "-lrt",
                                                               "-lpthread"]
        run(cmd)
    if force or _fast_stale():
        run(_fast_command(cc))
        with open(FAST_FOR, "w") as f:
            f.write(_fast_made_for())
    return LIB


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("-v", "--verbose", action="store_true")
    ap.add_argument("--ptxas", action="store_true", help="print ptxas register/smem usage")
    a = ap.parse_args()
    print(build(a.force, a.verbose, a.ptxas))
