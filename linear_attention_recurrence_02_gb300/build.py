"""Build libkda.so in-tree with nvcc for sm_103a.

Each ``csrc/*.cu`` is compiled in parallel to an object file, then linked
into ``_build/libkda.so`` (CUDA runtime linked statically, no other
dependencies). ``csrc/kda_fastcall.c``, the host side of the 8-bit operators'
binding, is compiled by the C compiler into ``_build/kda_fastcall.<abi>.so``, a
CPython extension. Nothing is installed outside the source tree.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import shlex
import shutil
import subprocess
import sysconfig
import warnings

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(BUILD, "libkda.so")
# the suffix names the interpreter's version and the machine: another Python builds its own
FASTCALL = os.path.join(BUILD, "kda_fastcall" + (sysconfig.get_config_var("EXT_SUFFIX") or ".so"))
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "--expt-relaxed-constexpr",
              "-Xcompiler", "-fPIC", "-Xptxas", "-v"] + ARCH


def _nvcc():
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", shutil.which("nvcc")):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _newer(out, deps) -> bool:
    return os.path.exists(out) and all(os.path.getmtime(p) <= os.path.getmtime(out) for p in deps)


def _library_up_to_date() -> bool:
    return _newer(LIB, [*glob.glob(os.path.join(CSRC, "*.cu")), *glob.glob(os.path.join(CSRC, "*.cuh")),
                        os.path.join(INCLUDE, "kda.h")])


def _fastcall_up_to_date() -> bool:
    return _newer(FASTCALL, glob.glob(os.path.join(CSRC, "*.c")))


def up_to_date() -> bool:
    return _library_up_to_date() and _fastcall_up_to_date()


def _compile_fastcall():
    cc = shlex.split(os.environ.get("CC", "")) or [c for c in (shutil.which("gcc"), shutil.which("cc")) if c][:1]
    if not cc:
        raise RuntimeError("no C compiler found")
    src, out = os.path.join(CSRC, "kda_fastcall.c"), FASTCALL + f".tmp{os.getpid()}"
    r = subprocess.run([*cc, "-O2", "-std=c11", "-Wall", "-shared", "-fPIC", "-I", sysconfig.get_paths()["include"],
                        src, "-o", out], capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{cc[0]} failed for {src}:\n{r.stdout}\n{r.stderr}")
    os.replace(out, FASTCALL)


def build_library(force: bool = False, verbose: bool = False) -> str:
    """Compile every csrc/*.cu for sm_103a and link libkda.so; returns its path. The Python extension is
    built beside it; the library does without, so where that fails there is a warning."""
    os.makedirs(BUILD, exist_ok=True)
    with cf.ThreadPoolExecutor(max_workers=8) as ex:
        host = ex.submit(_compile_fastcall) if force or not _fastcall_up_to_date() else None
        if force or not _library_up_to_date():
            _compile_library(ex, verbose)
        if host is not None:
            try:
                host.result()
            except (RuntimeError, OSError) as e:
                warnings.warn(f"{os.path.basename(FASTCALL)} was not built (it needs a C compiler and Python.h); "
                              f"the Python binding of the 8-bit operators will not work: {e}")
    return LIB


def _compile_library(ex, verbose):
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

    objs = list(ex.map(compile_one, srcs))
    tmp = LIB + f".tmp{os.getpid()}"
    r = subprocess.run([nvcc, *ARCH, "-shared", "-o", tmp, *objs], capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    if verbose:
        for o in objs:
            print(open(o + ".ptxas.txt").read())


if __name__ == "__main__":
    print(build_library(force=True, verbose=True))
