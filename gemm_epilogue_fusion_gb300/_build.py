"""Builds the sm_103a shared library ``libcoda_gb300.so`` in-tree with nvcc.

Each CUDA translation unit compiles in parallel to an object, then the objects
link into one shared library exporting the C ABI of ``include/coda.h``.
The argument marshalling of the short calls (coda_marshal.c) is a CPython
extension module beside it, named for the running interpreter.  The binding
does without it (its Python checks serve every call), so where it cannot be
compiled, a Python without headers for one, that is a warning.
Rebuilds only what a source, header or this script is newer than.
"""
from __future__ import annotations

import concurrent.futures as cf
import contextlib
import os
import shutil
import subprocess
import sysconfig
import warnings

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libcoda_gb300.so")
MARSHAL = os.path.join(PKG, "_coda_marshal" + (sysconfig.get_config_var("EXT_SUFFIX") or ".so"))

SOURCES = ["coda_gemm_bf16.cu", "coda_gemm_tf32.cu", "coda_gemm_e4m3.cu", "coda_aux.cu", "coda_paged.cu",
           "coda_logprobs.cu", "coda_abi.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc() -> str:
    cand = os.environ.get("NVCC") or shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found: the CUDA library cannot be built")
    return cand


def _flags(extra=()):
    return ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
                   "-I", CSRC, "-I", INCLUDE, "--expt-relaxed-constexpr", *extra]


def _inputs():
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC)]
    files += [os.path.join(INCLUDE, f) for f in os.listdir(INCLUDE)]
    files.append(os.path.abspath(__file__))
    return files


def up_to_date() -> bool:
    if not os.path.exists(LIB):
        return False
    t = os.path.getmtime(LIB)
    return all(os.path.getmtime(f) <= t for f in _inputs())


def marshal_up_to_date() -> bool:
    if not os.path.exists(MARSHAL):
        return False
    t = os.path.getmtime(MARSHAL)
    files = [os.path.join(CSRC, "coda_marshal.c"), os.path.join(INCLUDE, "coda.h"), os.path.abspath(__file__)]
    return all(os.path.getmtime(f) <= t for f in files)


def build_marshal() -> None:
    """The extension module of coda_marshal.c, for the running Python.  Where it cannot be compiled: a warning, and none
    is left (one of other sources would pass other arguments)."""
    tmp = MARSHAL + f".tmp{os.getpid()}"
    try:
        cuda_include = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc()))), "include")
        cmd = [os.environ.get("CC") or "gcc", "-O2", "-fPIC", "-shared", "-std=gnu11", "-fvisibility=hidden", "-Wall",
               "-I", sysconfig.get_paths()["include"], "-I", INCLUDE, "-isystem", cuda_include,
               os.path.join(CSRC, "coda_marshal.c"), "-o", tmp]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"{cmd[0]} failed:\n{r.stdout}\n{r.stderr}")
        os.replace(tmp, MARSHAL)
    except (OSError, RuntimeError) as e:
        with contextlib.suppress(OSError):
            os.remove(MARSHAL)
        warnings.warn(f"coda_marshal.c could not be compiled, the decode and scoring calls take longer on the host: {e}",
                      RuntimeWarning, stacklevel=3)


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    """Compile and link what is out of date; returns the library path.  Raises on compiler errors (of the library)."""
    if force or extra_flags or not up_to_date():
        _build_library(verbose, extra_flags)
    if force or not marshal_up_to_date():
        build_marshal()
    return LIB


def _build_library(verbose, extra_flags) -> None:
    os.makedirs(BUILD, exist_ok=True)
    cc = nvcc()

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
        cmd = [cc, *_flags(extra_flags), "-c", os.path.join(CSRC, src), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            print(r.stdout, r.stderr)
        return obj

    with cf.ThreadPoolExecutor(max_workers=len(SOURCES)) as ex:
        objs = list(ex.map(compile_one, SOURCES))
    tmp = LIB + f".tmp{os.getpid()}"
    # The shared CUDA runtime: inside a PyTorch process the already-loaded
    # libcudart.so.13 is reused, so the library and torch agree on the
    # current device and share streams; rpath covers standalone use.
    cuda_lib = os.path.join(os.path.dirname(os.path.dirname(cc)), "lib64")
    cmd = [cc, *ARCH, "-shared", "-cudart", "shared", "-o", tmp, *objs, "-Xlinker", f"-rpath,{cuda_lib}"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)


if __name__ == "__main__":
    import sys
    print(build(force="--force" in sys.argv, verbose=True))
