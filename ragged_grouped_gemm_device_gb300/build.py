"""Build libmoe_gg.so in place: every .cu under csrc/ compiled for sm_103a by nvcc, in parallel,
then linked into one shared library next to this file. Rebuilds only when a source or header is
newer than the library (or when forced).

build(debug=True) compiles the same sources with -DMOE_GG_DEBUG into libmoe_gg_debug.so (same
ABI): device-side bounds checks at the data-dependent global accesses and a wait for the stream
at the end of every entry point, read back with moe_debug_report().

build_binding() compiles csrc/binding.cpp, the CPython extension that marshals the calls of a decode
step, next to this file; where it cannot be built (no C++ compiler, no headers of Python or torch, a failing
compile) the ctypes binding does it."""
from __future__ import annotations

import concurrent.futures as cf
import glob
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libmoe_gg.so")
DEBUG_LIB = os.path.join(PKG, "libmoe_gg_debug.so")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall",
         "--expt-relaxed-constexpr", "-I", os.path.join(ROOT, "include")]


def nvcc() -> str:
    path = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(path):
        raise RuntimeError("nvcc not found")
    return path


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _inputs():
    return sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) + \
        glob.glob(os.path.join(ROOT, "include", "*.h")) + [os.path.abspath(__file__)]


def up_to_date(lib: str = LIB) -> bool:
    if not os.path.exists(lib):
        return False
    t = os.path.getmtime(lib)
    return all(os.path.getmtime(p) <= t for p in _inputs())


def build(force: bool = False, verbose: bool = False, extra_flags=(), debug: bool = False) -> str:
    lib = DEBUG_LIB if debug else LIB
    if not force and up_to_date(lib):
        return lib
    objdir = os.path.join(BUILD, "debug") if debug else BUILD
    os.makedirs(objdir, exist_ok=True)
    cc = nvcc()
    if debug:
        extra_flags = (*extra_flags, "-DMOE_GG_DEBUG")

    def compile_one(src):
        obj = os.path.join(objdir, os.path.basename(src) + ".o")
        cmd = [cc, *ARCH, *FLAGS, *extra_flags, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            print(r.stdout, r.stderr)
        return obj

    srcs = sources()
    with cf.ThreadPoolExecutor(max_workers=max(1, min(len(srcs), os.cpu_count() or 4))) as ex:
        objs = list(ex.map(compile_one, srcs))
    tmp = lib + ".tmp"
    cmd = [cc, *ARCH, "-shared", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, lib)
    return lib


BINDING = os.path.join(PKG, "_binding.so")


def build_binding(force: bool = False):
    """Path of the CPython extension, or None where it cannot be built: without torch, a compiler or headers, or
    when the compile fails, which is printed. An extension of older sources does not stay behind then."""
    src = os.path.join(CSRC, "binding.cpp")
    spec = importlib.util.find_spec("torch")
    if spec is None or spec.origin is None:
        return None
    torch = os.path.dirname(spec.origin)
    deps = [src, os.path.join(ROOT, "include", "moe_gg.h"), os.path.abspath(__file__), os.path.join(torch, "version.py")]
    if not force and os.path.exists(BINDING) and all(os.path.getmtime(p) <= os.path.getmtime(BINDING) for p in deps):
        return BINDING
    cc, inc = shutil.which("g++") or shutil.which("c++"), sysconfig.get_paths()["include"]
    if cc is None or not os.path.exists(os.path.join(inc, "Python.h")):
        return _without_binding()
    cuda = os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include")
    lib = os.path.join(torch, "lib")
    tmp = BINDING + ".tmp"
    cmd = [cc, "-O2", "-std=c++17", "-Wall", "-shared", "-fPIC", "-I", inc, "-I", os.path.join(torch, "include"), "-I",
           os.path.join(torch, "include", "torch", "csrc", "api", "include"), "-I", cuda, src, "-o", tmp, "-L", lib,
           "-Wl,-rpath," + lib, "-ltorch_python", "-ltorch_cpu", "-lc10_cuda", "-lc10"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        print(f"{cc} failed for {src}, the ctypes binding is used:\n{r.stdout}\n{r.stderr}", file=sys.stderr)
        return _without_binding()
    os.replace(tmp, BINDING)
    return BINDING


def _without_binding():
    if os.path.exists(BINDING):
        os.remove(BINDING)


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True, debug="--debug" in sys.argv))
    print(build_binding(force="--force" in sys.argv))
