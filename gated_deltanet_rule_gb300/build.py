"""Builds libgdr.so in-tree from csrc/*.cu for sm_103a (nvcc, one -gencode, parallel compiles) and the
compiled Python binding _gdr_bind.so from csrc/gdr_bind.cpp (g++, against torch's headers).

Usage: python -m gated_deltanet_rule_gb300.build [--force] [--verbose]
Objects go to gated_deltanet_rule_gb300/_build/, the library to gated_deltanet_rule_gb300/libgdr.so.
"""
from __future__ import annotations

import glob
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
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libgdr.so")
BIND = os.path.join(PKG, "_gdr_bind.so")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC,-O2",
                     "--expt-relaxed-constexpr", "-I", INCLUDE, "-I", CSRC]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def bind_commands(obj: str, out: str) -> tuple[list[str], list[str]]:
    """g++ commands that compile the binding and link it against torch's libraries and libgdr.so."""
    torch = os.path.dirname(importlib.util.find_spec("torch").origin)
    cuda = os.path.dirname(os.path.dirname(nvcc()))
    dirs = [sysconfig.get_paths()["include"], os.path.join(torch, "include"),
            os.path.join(torch, "include", "torch", "csrc", "api", "include"), os.path.join(cuda, "include")]
    cc = ["g++", "-c", os.path.join(CSRC, "gdr_bind.cpp"), "-o", obj, "-O2", "-fPIC", "-std=c++17", "-I", INCLUDE]
    for d in dirs:
        cc += ["-isystem", d]
    ld = ["g++", "-shared", obj, "-o", out, "-L" + os.path.join(torch, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10",
          "-lc10_cuda", "-L" + PKG, "-l:libgdr.so", "-Wl,-rpath,$ORIGIN"]
    return cc, ld


def _stale(target: str, deps: list[str]) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def build(force: bool = False, verbose: bool = False, extra_flags: list[str] | None = None) -> str:
    os.makedirs(BUILD, exist_ok=True)
    srcs = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    headers = sorted(glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(CSRC, "*.cuh")) +
                     glob.glob(os.path.join(INCLUDE, "*.h")))
    flags = NVCC_FLAGS + list(extra_flags or [])
    jobs = []
    objs = []
    for src in srcs:
        obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
        objs.append(obj)
        if force or _stale(obj, [src] + headers + [__file__]):
            jobs.append([nvcc(), "-c", src, "-o", obj] + flags)

    bind_obj = os.path.join(BUILD, "gdr_bind.o")
    bind_cc, bind_ld = bind_commands(bind_obj, BIND + f".tmp{os.getpid()}")
    if force or _stale(bind_obj, [os.path.join(CSRC, "gdr_bind.cpp"), os.path.join(INCLUDE, "gdr.h"), __file__]):
        jobs.append(bind_cc)

    def run(cmd):
        if verbose:
            print(" ".join(cmd), flush=True)
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"{os.path.basename(cmd[0])} failed:\n{' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            print(r.stdout + r.stderr, flush=True)

    if jobs:
        with ThreadPoolExecutor(max_workers=max(1, len(jobs))) as ex:
            list(ex.map(run, jobs))
    if force or jobs or _stale(LIB, objs):
        tmp = LIB + f".tmp{os.getpid()}"
        run([nvcc(), "-shared", "-o", tmp] + objs + ARCH + ["-Xcompiler", "-fPIC"])
        os.replace(tmp, LIB)
    if force or _stale(BIND, [bind_obj]):
        run(bind_ld)
        os.replace(BIND + f".tmp{os.getpid()}", BIND)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="--verbose" in sys.argv))
