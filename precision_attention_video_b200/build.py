"""Build libtiered_attn.so (sm_100a) in-tree with nvcc.

Each CUDA source is compiled to an object in parallel, then linked into a
shared library next to this file; the CUDA runtime is linked statically so
the library needs nothing beyond the driver at run time.  The C++ entry of the
cached-attention operators (_cache_call.so) is compiled by the host compiler
against the installed torch; where its headers are missing the library is built
all the same, and cache.py marshals the calls itself.
"""

from __future__ import annotations

import os
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(HERE, "libtiered_attn.so")
CALL = os.path.join(HERE, "_cache_call.so")

SOURCES = ["ta_api.cu", "ta_prep.cu", "ta_route.cu", "ta_attn.cu", "ta_attn2.cu", "ta_static.cu",
           "ta_cache_api.cu", "ta_cache.cu", "ta_cache_attn.cu"]
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
         "-I", INCLUDE, "-I", CSRC]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", "nvcc"):
        if cand and (os.path.sep not in cand or os.path.exists(cand)):
            return cand
    return "nvcc"


def _deps_mtime() -> float:
    paths = [os.path.join(CSRC, f) for f in os.listdir(CSRC)]
    paths += [os.path.join(INCLUDE, f) for f in os.listdir(INCLUDE)]
    paths.append(os.path.abspath(__file__))
    return max(os.path.getmtime(p) for p in paths)


def _build_call() -> None:
    """Compile _cache_call.so."""
    import sysconfig

    import torch
    root = os.path.join(os.path.dirname(torch.__file__))
    cuda = os.path.dirname(os.path.dirname(nvcc())) if os.path.sep in nvcc() else "/usr/local/cuda"
    inc = [os.path.join(root, "include"), os.path.join(root, "include", "torch", "csrc", "api", "include"),
           os.path.join(cuda, "include"), sysconfig.get_paths()["include"]]
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", "-I", INCLUDE,
           *[x for i in inc for x in ("-isystem", i)],
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           os.path.join(CSRC, "ta_cache_py.cpp"), "-o", CALL + ".tmp",
           "-L" + os.path.join(root, "lib"), "-lc10", "-lc10_cuda", "-ltorch_python"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode:
        sys.stderr.write(r.stdout + r.stderr)
        raise RuntimeError("compiler failed on ta_cache_py.cpp")
    os.replace(CALL + ".tmp", CALL)


def build(force: bool = False, verbose: bool = False, ptxas_verbose: bool = False) -> str:
    """Compile and link the library if any source is newer than it; return its path."""
    deps = _deps_mtime()
    _build_lib(deps, force, verbose, ptxas_verbose)
    if force or not os.path.exists(CALL) or os.path.getmtime(CALL) < deps:
        try:
            _build_call()
        except (RuntimeError, OSError, ImportError) as e:
            # (an old one would not match the library)
            if os.path.exists(CALL):
                os.remove(CALL)
            sys.stderr.write(f"_cache_call.so is not built ({e}): cached attention is called through "
                             "ctypes, some 10 us a call slower\n")
    return LIB


def _build_lib(deps: float, force: bool, verbose: bool, ptxas_verbose: bool) -> None:
    if not force and os.path.exists(LIB) and os.path.getmtime(LIB) >= deps:
        return
    os.makedirs(BUILD, exist_ok=True)
    extra = ["-Xptxas", "-v"] if ptxas_verbose else []

    def compile_one(src: str) -> str:
        obj = os.path.join(BUILD, src.replace(".cu", ".o"))
        cmd = [nvcc(), *ARCH, *FLAGS, *extra, "-c", os.path.join(CSRC, src), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if verbose or ptxas_verbose or r.returncode:
            sys.stderr.write(r.stdout + r.stderr)
        if r.returncode:
            raise RuntimeError(f"nvcc failed on {src}")
        return obj

    with ThreadPoolExecutor(max_workers=len(SOURCES)) as ex:
        objs = list(ex.map(compile_one, SOURCES))
    tmp = LIB + ".tmp"
    cmd = [nvcc(), *ARCH, "-shared", "-cudart", "static", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode:
        sys.stderr.write(r.stdout + r.stderr)
        raise RuntimeError("link failed")
    os.replace(tmp, LIB)


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True, ptxas_verbose="-v" in sys.argv)
    print(LIB)
