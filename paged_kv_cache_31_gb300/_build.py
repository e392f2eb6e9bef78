"""Build libpa.so (CUDA, sm_103a) in-tree with nvcc.

Each translation unit under csrc/ is compiled in parallel with
``-gencode arch=compute_103a,code=sm_103a`` and linked into
``paged_kv_cache_31_gb300/libpa.so`` (static CUDA runtime; the driver's tensor-map
encoder is reached through cudaGetDriverEntryPointByVersion, so libcuda is not linked).
csrc/pa_calls.cpp (host code over torch's C++ headers) becomes the Python module ``_calls`` next to
it, which is linked to libpa.so.  Its file name holds the Python and torch that it was compiled
for, so it is built anew, and no other one is loaded, after either has changed.
"""
from __future__ import annotations

import concurrent.futures
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libpa.so")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
         "-I", INCLUDE, "-I", CSRC]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def calls_path() -> str:
    """The module _calls of this Python and torch."""
    import torch

    return os.path.join(PKG, f"_calls.{sysconfig.get_config_var('SOABI')}-torch{torch.__version__}.so")


def _newer(target: str, deps) -> bool:
    return os.path.exists(target) and all(
        os.path.getmtime(p) <= os.path.getmtime(target) for p in deps)


def lib_up_to_date() -> bool:
    headers = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cuh")]
    return _newer(LIB, [*sources(), *headers, os.path.join(INCLUDE, "pa.h")])


def calls_up_to_date() -> bool:
    return _newer(calls_path(), [os.path.join(CSRC, "pa_calls.cpp"), os.path.join(INCLUDE, "pa.h")])


def up_to_date() -> bool:
    return lib_up_to_date() and calls_up_to_date()


def _compile_calls(nvcc: str) -> str:
    import torch

    obj = os.path.join(BUILD, "pa_calls.o")
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc))), "include")
    inside = os.path.join(os.path.dirname(torch.__file__), "include")
    inc = [sysconfig.get_paths()["include"], inside, cuda]
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-Wall",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           "-I", INCLUDE, *(f for i in inc for f in ("-isystem", i)),
           "-c", os.path.join(CSRC, "pa_calls.cpp"), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on pa_calls.cpp:\n{r.stdout}\n{r.stderr}")
    return obj


def _link_calls(obj: str) -> None:
    import torch

    path = calls_path()
    tmp = path + f".tmp{os.getpid()}"
    libs = ["-L", os.path.join(os.path.dirname(torch.__file__), "lib")]
    cmd = ["g++", "-shared", "-o", tmp, obj, "-L", PKG, "-l:libpa.so", "-Wl,-rpath,$ORIGIN", *libs,
           "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, path)
    for f in os.listdir(PKG):  # those of another torch
        if f.startswith("_calls") and f.endswith(".so") and f != os.path.basename(path):
            os.remove(os.path.join(PKG, f))


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    lib, calls = force or not lib_up_to_date(), force or not calls_up_to_date()
    if not (lib or calls):
        return LIB
    nvcc = _nvcc()
    os.makedirs(BUILD, exist_ok=True)
    srcs = sources() if lib else []

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
        cmd = [nvcc, *ARCH, *FLAGS, *extra_flags, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            sys.stderr.write(r.stdout + r.stderr)
        return obj

    workers = max(1, min(len(srcs) + 1, os.cpu_count() or 4))
    with concurrent.futures.ThreadPoolExecutor(max_workers=workers) as ex:
        calls_obj = ex.submit(_compile_calls, nvcc) if calls else None
        objs = list(ex.map(compile_one, srcs))
        if lib:
            tmp = LIB + f".tmp{os.getpid()}"
            cmd = [nvcc, *ARCH, "-shared", "-o", tmp, *objs]
            r = subprocess.run(cmd, capture_output=True, text=True)
            if r.returncode != 0:
                raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
            os.replace(tmp, LIB)
        if calls:
            _link_calls(calls_obj.result())
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True,
                extra_flags=["-Xptxas", "-v"] if "--ptxas-v" in sys.argv else []))
