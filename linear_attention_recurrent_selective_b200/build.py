"""Build libssu.so (the C-ABI CUDA library) in-tree for sm_100a with nvcc.

Usage: python -m linear_attention_recurrent_selective_b200.build [--force] [--verbose]
Objects go to _build/ at the repository root; the shared library lands next to this
file so that it travels with the package.

The Python binding's native argument marshalling (csrc/marshal.cpp, a CPython module that
reads torch tensors) is built beside it with the C++ compiler, under a name that says which
torch and which Python it was built against (_marshal.<torch>.<python>.so): it reads their
objects, and is of no use to others. The library does not need it: where it cannot be built
(no C++ compiler, a torch without CUDA) the library is built all the same, with a warning.

The same sources also build libssu_waittest.so (objects in _build/waittest/), with
SSU_WAIT_TEST defined: the test suite's library in which a chosen bounded wait can be
made to run out (include/ssu_wait_test.h). Nothing but the tests loads it.
"""

from __future__ import annotations

import argparse
import concurrent.futures
import glob
import os
import shutil
import subprocess
import sys
import sysconfig
import warnings

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libssu.so")
WAITTEST_LIB = os.path.join(PKG, "libssu_waittest.so")

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall",
              "--expt-relaxed-constexpr", "-I", INCLUDE, "-I", CSRC] + ARCH


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libssu.so")


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return (sources() + glob.glob(os.path.join(CSRC, "*.cuh")) +
            glob.glob(os.path.join(INCLUDE, "*.h")))


def up_to_date(lib: str = LIB) -> bool:
    if not os.path.exists(lib):
        return False
    t = os.path.getmtime(lib)
    return all(os.path.getmtime(p) <= t for p in _deps() + [__file__])


def marshal_path() -> str:
    """Where the binding's native module for this torch and this Python is."""
    import torch
    tag = sysconfig.get_config_var("EXT_SUFFIX")
    return os.path.join(PKG, f"_marshal.{torch.__version__}{tag}")


def build_marshal(force: bool = False) -> str:
    """Build the binding's native argument marshalling."""
    import torch
    src, out = os.path.join(CSRC, "marshal.cpp"), marshal_path()
    deps = [src, __file__] + glob.glob(os.path.join(INCLUDE, "*.h"))
    if not force and os.path.exists(out) and \
            all(os.path.getmtime(p) <= os.path.getmtime(out) for p in deps):
        return out
    home = os.path.dirname(torch.__file__)
    inc, libs = os.path.join(home, "include"), os.path.join(home, "lib")
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc()))), "include")
    tmp = out + ".tmp"
    cmd = [shutil.which("g++") or "g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", "-I", INCLUDE,
           "-isystem", inc, "-isystem", os.path.join(inc, "torch", "csrc", "api", "include"),
           "-isystem", sysconfig.get_paths()["include"], "-isystem", cuda, src, "-o", tmp,
           "-L", libs, f"-Wl,-rpath,{libs}", "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on {src}:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, out)
    return out


def build(force: bool = False, verbose: bool = False, waittest: bool = False) -> str:
    """Build libssu.so and, where that can be done, the binding's native module (or, with
    waittest, the test library libssu_waittest.so)."""
    lib = WAITTEST_LIB if waittest else LIB
    if force or not up_to_date(lib):
        _build_library(lib, verbose, waittest)
    if not waittest:
        try:
            build_marshal(force)
        except (ImportError, OSError, RuntimeError) as e:
            warnings.warn(f"libssu.so is built, the binding's native module is not: {e}",
                          stacklevel=2)
    return lib


def _build_library(lib: str, verbose: bool, waittest: bool) -> None:
    objdir = os.path.join(BUILD, "waittest") if waittest else BUILD
    os.makedirs(objdir, exist_ok=True)
    cc = nvcc()
    extra = ["-Xptxas", "-v"] if verbose else []
    if waittest:
        extra += ["-DSSU_WAIT_TEST"]

    def compile_one(src):
        obj = os.path.join(objdir, os.path.basename(src) + ".o")
        cmd = [cc, *NVCC_FLAGS, *extra, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        if verbose:
            sys.stderr.write(r.stderr)
        return obj

    with concurrent.futures.ThreadPoolExecutor(max_workers=os.cpu_count() or 4) as ex:
        objs = list(ex.map(compile_one, sources()))
    tmp = lib + ".tmp"
    cmd = [cc, *ARCH, "-shared", "-cudart", "static", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, lib)


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--verbose", action="store_true", help="print ptxas register/spill info")
    ap.add_argument("--waittest", action="store_true",
                    help="build the test library libssu_waittest.so instead")
    args = ap.parse_args()
    print(build(force=args.force, verbose=args.verbose, waittest=args.waittest))
