"""In-tree build of libchain_gb300.so for sm_103a (nvcc, no cmake).

Each translation unit under csrc/ compiles in parallel to an object file in
chain_gb300/_build/, then nvcc links the shared library beside this file.
Rebuilds only what changed (sources or the shared headers).  binding.c, the
CPython entry to the library's small calls, is compiled with gcc into
chain_gb300/_native and linked to the library beside it; where Python's headers
or gcc are missing the library stands alone, and those calls say so.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import shutil
import subprocess
import sysconfig
import warnings

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libchain_gb300.so")
NATIVE = os.path.join(HERE, "_native" + sysconfig.get_config_var("EXT_SUFFIX"))
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-O2",
         "--expt-relaxed-constexpr", "-I", os.path.join(ROOT, "include")]


def _nvcc() -> str:
    for c in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if c and os.path.exists(c):
            return c
    raise RuntimeError("chain_gb300: nvcc not found; the CUDA library cannot be built")


def _headers():
    return glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) + \
        glob.glob(os.path.join(ROOT, "include", "*.h"))


def _run(cmd, verbose=False):
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"compilation failed:\n{' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    if verbose and (r.stdout or r.stderr):
        print(r.stdout + r.stderr)


def build_native(force: bool = False, verbose: bool = False) -> str:
    """The CPython module, once the library is there."""
    src = os.path.join(CSRC, "binding.c")
    newest = max(os.path.getmtime(f) for f in [src, *_headers()])
    if not force and os.path.exists(NATIVE) and os.path.getmtime(NATIVE) >= newest:
        return NATIVE
    include = sysconfig.get_paths()["include"]
    if not os.path.exists(os.path.join(include, "Python.h")):
        raise RuntimeError(f"chain_gb300: no Python.h in {include}; the native module cannot be built")
    if not shutil.which("gcc"):
        raise RuntimeError("chain_gb300: gcc not found; the native module (Python.h) cannot be built")
    tmp = NATIVE + f".tmp{os.getpid()}"
    _run(["gcc", "-O2", "-std=c11", "-Wall", "-fPIC", "-shared", "-I", include, src, "-o", tmp, "-L" + HERE,
          "-lchain_gb300", "-Wl,-rpath,$ORIGIN"], verbose)
    os.replace(tmp, NATIVE)
    return NATIVE


def build(force: bool = False, verbose: bool = False, extra=()) -> str:
    os.makedirs(BUILD, exist_ok=True)
    nvcc = _nvcc()
    srcs = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    hdr_t = max((os.path.getmtime(h) for h in _headers()), default=0.0)
    jobs = []
    objs = []
    for s in srcs:
        o = os.path.join(BUILD, os.path.basename(s)[:-3] + ".o")
        objs.append(o)
        if force or not os.path.exists(o) or os.path.getmtime(o) < max(os.path.getmtime(s), hdr_t):
            jobs.append([nvcc, *ARCH, *FLAGS, *extra, "-c", s, "-o", o])

    def run(cmd):
        _run(cmd, verbose)

    if jobs:
        with cf.ThreadPoolExecutor(max_workers=min(len(jobs), os.cpu_count() or 4)) as ex:
            list(ex.map(run, jobs))
    stale = (not os.path.exists(LIB) or jobs or
             os.path.getmtime(LIB) < max(os.path.getmtime(o) for o in objs))
    if force or stale:
        tmp = LIB + f".tmp{os.getpid()}"
        run([nvcc, *ARCH, "-shared", "-Xlinker", "-soname=" + os.path.basename(LIB), "-o", tmp, *objs])
        os.replace(tmp, LIB)
    if shutil.which("gcc") and os.path.exists(os.path.join(sysconfig.get_paths()["include"], "Python.h")):
        build_native(force, verbose)
    else:
        warnings.warn("chain_gb300: built without its native module, which needs gcc and Python.h: the norm, "
                      "rotation and paged cache calls are there from C only", RuntimeWarning, stacklevel=2)
    return LIB


if __name__ == "__main__":
    import sys
    print(build(force="--force" in sys.argv, verbose=True,
                extra=["-Xptxas", "-v"] if "--ptxas-v" in sys.argv else []))
