"""Build libkda.so in-tree with nvcc for sm_100a (B200).

    python -m gated_delta_rule_155_b200.build [--force] [-j N]

Each ``csrc/*.cu`` is compiled separately (in parallel) with
``-gencode arch=compute_100a,code=sm_100a -O3 -lineinfo`` and linked into
``gated_delta_rule_155_b200/libkda.so`` (CUDA runtime linked statically).
Objects go to ``_build/`` at the repository root.  ``csrc/calls.cpp``, the binding's short
calls, is compiled with g++ against torch's headers into an extension module whose file name has
the versions of torch and Python; where that fails, the library is built all the same, with a warning.
A rebuild happens only when a source or header is newer than the library.
"""
from __future__ import annotations

import argparse
import glob
import os
import shutil
import subprocess
import sys
import sysconfig
import warnings
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
OBJ_DIR = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libkda.so")

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
CFLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-O3",
          "--expt-relaxed-constexpr", "-I", INCLUDE, "-I", CSRC]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libkda.so")


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) + \
        glob.glob(os.path.join(INCLUDE, "*.h")) + [os.path.abspath(__file__)]


def up_to_date() -> bool:
    if not os.path.exists(LIB):
        return False
    t = os.path.getmtime(LIB)
    return all(os.path.getmtime(d) <= t for d in _deps())


def _newer(lib, deps) -> bool:
    return os.path.exists(lib) and all(os.path.getmtime(d) <= os.path.getmtime(lib) for d in deps)


def _abi() -> int:
    import torch

    return int(torch._C._GLIBCXX_USE_CXX11_ABI)


def calls_path() -> str:
    """Where the short calls' module for this torch and this Python is.  It reads tensors through torch's C++ headers, so
    one that was built against others is another file, which is neither current nor loaded."""
    import torch

    return os.path.join(PKG, f"_calls.torch-{torch.__version__}-cxx{_abi()}.{sysconfig.get_config_var('SOABI')}.so")


def build_calls(force: bool = False, verbose: bool = False) -> str:
    src, calls = os.path.join(CSRC, "calls.cpp"), calls_path()
    if not force and _newer(calls, [src, os.path.join(INCLUDE, "kda.h"), os.path.abspath(__file__)]):
        return calls
    if os.path.exists(calls):
        os.remove(calls)          # it does not fit these sources: where the build fails, none is better than it
    import torch
    root = os.path.join(os.path.dirname(torch.__file__))
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))
    tmp = calls + f".tmp{os.getpid()}"
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared",
           f"-D_GLIBCXX_USE_CXX11_ABI={_abi()}", "-I", os.path.join(root, "include"),
           "-I", os.path.join(cuda, "include"), "-I", sysconfig.get_paths()["include"], src, "-o", tmp,
           "-L", os.path.join(root, "lib"), "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python"]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on calls.cpp:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, calls)
    return calls


def build(force: bool = False, jobs: int = 0, verbose: bool = False, extra=()) -> str:
    lib = build_library(force, jobs, verbose, extra)
    try:
        build_calls(force, verbose)
    except (RuntimeError, OSError, ImportError) as e:     # marshalling only: the library does without
        warnings.warn(f"the _calls extension was not built, short calls will be marshalled in Python: {e}", RuntimeWarning, stacklevel=2)
    return lib


def build_library(force: bool = False, jobs: int = 0, verbose: bool = False, extra=()) -> str:
    if not force and up_to_date():
        return LIB
    os.makedirs(OBJ_DIR, exist_ok=True)
    cc = nvcc()
    srcs = sources()

    def compile_one(src):
        obj = os.path.join(OBJ_DIR, os.path.basename(src) + ".o")
        cmd = [cc, *ARCH, *CFLAGS, *extra, "-c", src, "-o", obj]
        if verbose:
            print(" ".join(cmd), flush=True)
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {os.path.basename(src)}:\n{r.stdout}\n{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            print(r.stdout + r.stderr, flush=True)
        return obj

    with ThreadPoolExecutor(max_workers=jobs or min(8, len(srcs))) as ex:
        objs = list(ex.map(compile_one, srcs))
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [cc, *ARCH, "-shared", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    return LIB


def main(argv=None):
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("-j", type=int, default=0)
    ap.add_argument("-v", action="store_true")
    ap.add_argument("--ptxas-v", action="store_true", help="print register/spill/smem usage")
    a = ap.parse_args(argv)
    extra = ["-Xptxas", "-v"] if a.ptxas_v else []
    print(build(force=a.force or a.ptxas_v, jobs=a.j, verbose=a.v or a.ptxas_v, extra=extra))


if __name__ == "__main__":
    sys.exit(main())
