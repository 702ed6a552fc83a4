"""Build of the CUDA library ``libspecverify.so`` (sm_103a) next to this file.

Each translation unit is compiled by its own nvcc process (in parallel), then linked with the
shared CUDA runtime so that the library uses the runtime already loaded by the host process.
Beside it the host compiler builds ``_fastcall``, the Python module that marshals the short calls'
arguments (csrc/fastcall.cpp).  It only saves host time: where it cannot be built (no headers of
Python, say) the library is built without it.
"""
from __future__ import annotations

import concurrent.futures as cf
import importlib.machinery
import os
import shutil
import subprocess
import warnings

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libspecverify.so")
FASTCALL = os.path.join(PKG, "_fastcall" + importlib.machinery.EXTENSION_SUFFIXES[0])
BUILD_DIR = os.path.join(PKG, "_build")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def _nvcc():
    for c in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", shutil.which("nvcc")):
        if c and os.path.exists(c):
            return c
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libspecverify.so")


def sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def _deps():
    files = sources() + [os.path.join(CSRC, f) for f in os.listdir(CSRC)
                         if f.endswith((".cuh", ".h"))]
    files += [os.path.join(INCLUDE, f) for f in os.listdir(INCLUDE)]
    return files


def build_fastcall(force: bool = False) -> str | None:
    """The marshalling module, against the installed torch's headers; None, with a warning, where it
    cannot be built.  Made again when its sources, its compiler's command or torch change."""
    import sysconfig

    import torch

    src = os.path.join(CSRC, "fastcall.cpp")
    base = os.path.dirname(torch.__file__)
    try:
        cuda = os.path.dirname(os.path.dirname(_nvcc()))
    except RuntimeError:  # a module that is there needs no toolkit
        cuda = "/usr/local/cuda"
    cmd = [shutil.which("g++") or "c++", "-O2", "-std=c++17", "-fPIC", "-shared", src,
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           "-I", INCLUDE, "-I", os.path.join(base, "include"),
           "-I", os.path.join(base, "include", "torch", "csrc", "api", "include"),
           "-I", sysconfig.get_paths()["include"], "-I", os.path.join(cuda, "include"),
           "-L", os.path.join(base, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda"]
    made_by = " ".join([torch.__version__] + cmd)
    note = os.path.join(BUILD_DIR, os.path.basename(FASTCALL) + ".made_by")
    newest = max(os.path.getmtime(src), os.path.getmtime(os.path.join(INCLUDE, "specverify.h")))
    if not force and os.path.exists(FASTCALL) and os.path.getmtime(FASTCALL) >= newest:
        try:
            with open(note) as f:
                if f.read() == made_by:
                    return FASTCALL
        except OSError:
            pass
    os.makedirs(BUILD_DIR, exist_ok=True)
    tmp = FASTCALL + f".{os.getpid()}.tmp"
    try:
        res = subprocess.run(cmd + ["-o", tmp], capture_output=True, text=True)
        error = res.stderr if res.returncode else None
    except OSError as e:  # no compiler
        error = str(e)
    if error is not None:
        if os.path.exists(FASTCALL):  # made for something else
            os.remove(FASTCALL)
        warnings.warn(f"built without _fastcall, the host compiler failed on {src}:\n{error}",
                      RuntimeWarning)
        return None
    os.replace(tmp, FASTCALL)
    with open(note, "w") as f:
        f.write(made_by)
    return FASTCALL


def build(force: bool = False, verbose: bool = False) -> str:
    with cf.ThreadPoolExecutor(1) as ex:  # beside the CUDA sources
        fast = ex.submit(build_fastcall, force)
        lib = build_library(force, verbose)
        fast.result()
    return lib


def build_library(force: bool = False, verbose: bool = False) -> str:
    newest = max(os.path.getmtime(f) for f in _deps())
    if not force and os.path.exists(LIB) and os.path.getmtime(LIB) >= newest:
        return LIB
    nvcc = _nvcc()
    os.makedirs(BUILD_DIR, exist_ok=True)
    flags = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC,-O2",
                    "-I", INCLUDE, "-I", CSRC, "--expt-relaxed-constexpr"]
    if verbose:
        flags += ["-Xptxas", "-v"]

    def compile_one(src):
        obj = os.path.join(BUILD_DIR, os.path.basename(src) + ".o")
        cmd = [nvcc, "-c", src, "-o", obj] + flags
        res = subprocess.run(cmd, capture_output=True, text=True)
        if res.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{res.stderr}")
        return obj, res.stderr

    with cf.ThreadPoolExecutor(max_workers=max(1, min(8, os.cpu_count() or 1))) as ex:
        results = list(ex.map(compile_one, sources()))
    if verbose:
        for _, err in results:
            print(err)
    tmp = LIB + f".{os.getpid()}.tmp"
    cmd = [nvcc, "-shared", "-o", tmp] + [o for o, _ in results] + ARCH + ["-cudart", "shared"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"link failed:\n{res.stderr}")
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    import sys
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
