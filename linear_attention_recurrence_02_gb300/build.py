"""Build libkda.so in-tree with nvcc for sm_103a.

Each ``csrc/*.cu`` is compiled in parallel to an object file, then linked
into ``_build/libkda.so`` (CUDA runtime linked statically, no other
dependencies). ``csrc/kda_fastcall.c``, the host side of the 8-bit operators'
binding, is compiled by the C compiler into ``_build/kda_fastcall.so``, a
CPython extension. Nothing is installed outside the source tree.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import shutil
import subprocess
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(BUILD, "libkda.so")
FASTCALL = os.path.join(BUILD, "kda_fastcall.so")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "--expt-relaxed-constexpr",
              "-Xcompiler", "-fPIC", "-Xptxas", "-v"] + ARCH


def _nvcc():
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", shutil.which("nvcc")):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _deps():
    return sorted(glob.glob(os.path.join(CSRC, "*.c")) + glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cuh"))
                  + [os.path.join(INCLUDE, "kda.h")])


def up_to_date() -> bool:
    if not os.path.exists(LIB) or not os.path.exists(FASTCALL):
        return False
    t = min(os.path.getmtime(LIB), os.path.getmtime(FASTCALL))
    return all(os.path.getmtime(p) <= t for p in _deps())


def build_library(force: bool = False, verbose: bool = False) -> str:
    """Compile every csrc/*.cu for sm_103a and link libkda.so; returns its path."""
    if not force and up_to_date():
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    nvcc = _nvcc()
    srcs = sorted(glob.glob(os.path.join(CSRC, "*.cu")))

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
        cmd = [nvcc, *NVCC_FLAGS, "-I", INCLUDE, "-I", CSRC, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
        with open(obj + ".ptxas.txt", "w") as f:
            f.write(r.stderr)
        return obj

    def compile_fastcall():
        cc = next((c for c in (os.environ.get("CC"), shutil.which("gcc"), shutil.which("cc")) if c), None)
        if cc is None:
            raise RuntimeError("no C compiler found")
        src, out = os.path.join(CSRC, "kda_fastcall.c"), FASTCALL + f".tmp{os.getpid()}"
        r = subprocess.run([cc, "-O2", "-std=c11", "-Wall", "-shared", "-fPIC", "-I", sysconfig.get_paths()["include"],
                            src, "-o", out], capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"{cc} failed for {src}:\n{r.stdout}\n{r.stderr}")
        os.replace(out, FASTCALL)

    with cf.ThreadPoolExecutor(max_workers=min(8, len(srcs) + 1)) as ex:
        host = ex.submit(compile_fastcall)
        objs = list(ex.map(compile_one, srcs))
        host.result()
    tmp = LIB + f".tmp{os.getpid()}"
    r = subprocess.run([nvcc, *ARCH, "-shared", "-o", tmp, *objs], capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    if verbose:
        for o in objs:
            print(open(o + ".ptxas.txt").read())
    return LIB


if __name__ == "__main__":
    print(build_library(force=True, verbose=True))
