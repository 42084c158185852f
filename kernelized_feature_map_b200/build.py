"""Build libkata.so (the sm_100a CUDA library behind include/kata.h) in-tree.

    python -m kernelized_feature_map_b200.build [--force] [--verbose]

Every ``csrc/*.cu`` is compiled by nvcc for ``sm_100a`` only and linked into
``kernelized_feature_map_b200/libkata.so`` with the CUDA runtime linked
statically, so the library loads without a GPU or driver (for the symbol
checks) and needs only the driver on a GPU machine.  Only the C ABI symbols
are exported.  ``csrc/binding.cpp``, host code that calls it with torch
tensors, is compiled by g++ into ``_binding.so`` beside it.
"""
from __future__ import annotations

import argparse
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
BUILD_DIR = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libkata.so")
BINDING = os.path.join(PKG, "_binding.so")
BINDING_SRC = os.path.join(CSRC, "binding.cpp")
TRACE_LIB = os.path.join(PKG, "libkata_trace.so")

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
NVCC_FLAGS = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
                     "--expt-relaxed-constexpr", "-I", INCLUDE, "-I", CSRC]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return (_sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h"))
            + glob.glob(os.path.join(INCLUDE, "*.h")))


def up_to_date() -> bool:
    if not os.path.exists(LIB):
        return False
    t = os.path.getmtime(LIB)
    return all(os.path.getmtime(d) <= t for d in _deps())


def _torch_dir() -> str:
    return os.path.dirname(importlib.util.find_spec("torch").origin)


def binding_up_to_date() -> bool:
    """Newer than its sources and than the torch it was compiled against."""
    if not os.path.exists(BINDING):
        return False
    t = os.path.getmtime(BINDING)
    deps = [BINDING_SRC, os.path.join(INCLUDE, "kata.h"), os.path.join(_torch_dir(), "version.py")]
    return all(os.path.getmtime(d) <= t for d in deps)


def build_binding(force: bool = False, verbose: bool = False) -> str:
    """Compile _binding.so (csrc/binding.cpp, host code only) against the installed torch and libkata.so."""
    if not force and binding_up_to_date():
        return BINDING
    import torch
    inc, libs = os.path.join(_torch_dir(), "include"), os.path.join(_torch_dir(), "lib")
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc()))), "include")
    tmp = BINDING + ".tmp.%d" % os.getpid()
    # the system compiler, whose libstdc++ is the shared one that torch uses
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
           "-D_GLIBCXX_USE_CXX11_ABI=%d" % torch._C._GLIBCXX_USE_CXX11_ABI, "-I", INCLUDE]
    for d in (inc, os.path.join(inc, "torch", "csrc", "api", "include"), sysconfig.get_paths()["include"], cuda):
        cmd += ["-isystem", d]
    cmd += [BINDING_SRC, "-o", tmp, "-L", PKG, "-l:libkata.so", "-Wl,-rpath,$ORIGIN", "-L", libs, "-lc10", "-lc10_cuda",
            "-ltorch_cpu", "-ltorch_cuda", "-ltorch_python"]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("g++ failed on %s:\n%s%s" % (BINDING_SRC, r.stdout, r.stderr))
    os.replace(tmp, BINDING)
    return BINDING


def build(force: bool = False, verbose: bool = False, extra_flags=(), trace: bool = False) -> str:
    """Compile and link libkata.so, and _binding.so, if any source is newer; returns libkata's path.

    trace=True builds libkata_trace.so instead: the same sources with
    KATA_ENABLE_TRACE defined (per-CTA pipeline timestamps, see
    csrc/kata_trace.cuh).  It is a diagnostic build, never loaded by the
    package.
    """
    lib_path = TRACE_LIB if trace else LIB
    if not force and not trace and up_to_date():
        build_binding(verbose=verbose)
        return LIB
    build_dir = BUILD_DIR + ("_trace" if trace else "")
    if trace:
        extra_flags = tuple(extra_flags) + ("-DKATA_ENABLE_TRACE",)
    os.makedirs(build_dir, exist_ok=True)
    cc = nvcc()

    def compile_one(src):
        obj = os.path.join(build_dir, os.path.basename(src) + ".o")
        cmd = [cc, *NVCC_FLAGS, *extra_flags, "-c", src, "-o", obj]
        if verbose:
            print(" ".join(cmd), flush=True)
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError("nvcc failed on %s:\n%s%s" % (src, r.stdout, r.stderr))
        if verbose and (r.stdout or r.stderr):
            print(r.stdout + r.stderr, flush=True)
        return obj

    with ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 1)) as ex:
        objs = list(ex.map(compile_one, _sources()))
    tmp = lib_path + ".tmp.%d" % os.getpid()
    cmd = [cc, *ARCH, "-shared", "-cudart", "static", "-Xcompiler", "-fvisibility=hidden", "-o", tmp, *objs,
           "-lpthread", "-ldl", "-lrt"]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("link failed:\n%s%s" % (r.stdout, r.stderr))
    os.replace(tmp, lib_path)
    if not trace:
        build_binding(force=force, verbose=verbose)
    return lib_path


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--verbose", action="store_true")
    ap.add_argument("--ptxas-info", action="store_true", help="print registers/spills/shared memory per kernel")
    ap.add_argument("--trace", action="store_true", help="build the diagnostic libkata_trace.so")
    a = ap.parse_args(argv)
    extra = ["-Xptxas", "-v"] if a.ptxas_info else []
    print(build(force=a.force or a.ptxas_info, verbose=a.verbose or a.ptxas_info, extra_flags=extra, trace=a.trace))


if __name__ == "__main__":
    sys.exit(main())
