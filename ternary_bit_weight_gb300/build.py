"""Build libtern.so in-tree with nvcc for sm_103a (GB300).

Each ``csrc/*.cu`` file is compiled separately and in parallel, then linked
into ``_build/libtern.so`` against the shared CUDA runtime.  ``csrc/tern_python.c``
becomes an extension module of the interpreter that builds, beside it: the argument
marshalling of the calls made for single tokens.  Where Python's headers are not
installed it is left out, and the binding marshals with ctypes.  Rebuilds only what
a newer source or header asks for.
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
LIB = os.path.join(BUILD, "libtern.so")
PY_SRC = os.path.join(CSRC, "tern_python.c")
PY_LIB = os.path.join(BUILD, "_tern_python" + (sysconfig.get_config_var("EXT_SUFFIX") or ".so"))

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC,-O2,-Wall",
              "-I", INCLUDE, "-I", CSRC]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libtern")


def _cuda_lib_dir(nvcc: str) -> str:
    return os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc))), "lib64")


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _newer(target: str, deps) -> bool:
    """target is missing or older than one of deps."""
    return not os.path.exists(target) or any(os.path.getmtime(d) > os.path.getmtime(target) for d in deps)


def _headers():
    return glob.glob(os.path.join(INCLUDE, "*.h")) + [__file__]


def python_headers():
    """Folder of Python.h, or None where it is not installed."""
    path = sysconfig.get_paths()["include"]
    return path if os.path.exists(os.path.join(path, "Python.h")) else None


def build(force: bool = False, verbose: bool = False, ptxas_info: bool = False) -> str:
    """Compile and link libtern.so and the extension module; returns libtern.so's path."""
    if force or _newer(LIB, sources() + glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(CSRC, "*.cuh"))
                       + _headers()):
        _build_library(verbose, ptxas_info)
    if python_headers() and (force or _newer(PY_LIB, _headers() + [PY_SRC])):
        _build_python()
    return LIB


def _build_library(verbose: bool, ptxas_info: bool) -> None:
    nvcc = _nvcc()
    os.makedirs(BUILD, exist_ok=True)
    extra = ["-Xptxas", "-v"] if ptxas_info else []

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
        cmd = [nvcc, *ARCH, *NVCC_FLAGS, *extra, "-c", src, "-o", obj]
        res = subprocess.run(cmd, capture_output=True, text=True)
        if res.returncode != 0:
            raise RuntimeError(f"nvcc failed for {os.path.basename(src)}:\n{res.stdout}\n{res.stderr}")
        if verbose or ptxas_info:
            print(res.stdout + res.stderr)
        return obj

    srcs = sources()
    with cf.ThreadPoolExecutor(max_workers=max(1, min(len(srcs), os.cpu_count() or 1))) as ex:
        objs = list(ex.map(compile_one, srcs))
    tmp = LIB + f".tmp{os.getpid()}"
    libdir = _cuda_lib_dir(nvcc)
    cmd = [nvcc, *ARCH, "-shared", "-o", tmp, *objs, "-cudart", "shared",
           "-Xlinker", f"-rpath,{libdir}"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"link of libtern.so failed:\n{res.stdout}\n{res.stderr}")
    os.replace(tmp, LIB)


def _build_python() -> None:
    """The extension module, by nvcc's host compiler."""
    tmp = PY_LIB + f".tmp{os.getpid()}"
    cmd = [_nvcc(), "-shared", "-cudart", "none", "-Xcompiler", "-fPIC,-O2,-Wall", "-I", python_headers(), "-I", INCLUDE,
           PY_SRC, "-o", tmp, "-L", BUILD, "-Xlinker", "-l:libtern.so", "-Xlinker", "-rpath,$ORIGIN"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"nvcc failed for tern_python.c:\n{res.stdout}\n{res.stderr}")
    os.replace(tmp, PY_LIB)


if __name__ == "__main__":
    import sys
    print(build(force="--force" in sys.argv, verbose=True, ptxas_info="--ptxas" in sys.argv))
