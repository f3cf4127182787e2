"""Build libmoecache.so in-tree with nvcc for sm_103a, and _operators.so, which takes torch
tensors to its operators, with g++ (no cmake).

Each source compiles to an object in parallel, then one link each.  The outputs
sit next to this file so the in-tree libraries are the ones that load.  Where torch
is not installed there is nothing for _operators.so to take, and it is left out;
libmoecache.so needs no torch and is there even if _operators.so fails.
"""
from __future__ import annotations

import glob
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libmoecache.so")
HOST = os.path.join(HERE, "_operators.so")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-O3",
         "--expt-relaxed-constexpr", "-DNDEBUG"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def build(verbose: bool = False, ptxas_info: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    srcs = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    cc = nvcc()
    extra = ["-Xptxas", "-v"] if ptxas_info else []

    def compile_one(src: str) -> str:
        obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
        cmd = [cc, *ARCH, *FLAGS, *extra, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stderr}")
        if verbose or ptxas_info:
            sys.stderr.write(r.stderr)
        return obj

    def compile_host() -> str:
        from torch.utils.cpp_extension import include_paths
        obj = os.path.join(BUILD, "operators_host.o")
        inc = [*include_paths(), sysconfig.get_paths()["include"], os.path.join(os.path.dirname(os.path.dirname(cc)), "include")]
        cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-w", *(f"-I{i}" for i in inc), "-c",
               os.path.join(CSRC, "operators_host.cpp"), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"g++ failed for operators_host.cpp:\n{r.stderr}")
        return obj

    torch = importlib.util.find_spec("torch") is not None
    with ThreadPoolExecutor(max_workers=min(9, len(srcs) + 1)) as ex:
        host = ex.submit(compile_host) if torch else None
        objs = list(ex.map(compile_one, srcs))
    tmp = LIB + ".tmp"
    cmd = [cc, *ARCH, "-shared", "-cudart", "static", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stderr}")
    os.replace(tmp, LIB)
    if not torch:
        if os.path.exists(HOST):
            os.remove(HOST)        # another library's
        return LIB
    host_obj = host.result()
    from torch.utils.cpp_extension import library_paths
    libs = [f"-L{p}" for p in library_paths()]
    cmd = [os.environ.get("CXX", "g++"), "-shared", "-o", HOST + ".tmp", host_obj, f"-L{HERE}", "-l:libmoecache.so", "-Wl,-rpath,$ORIGIN",
           *libs, "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stderr}")
    os.replace(HOST + ".tmp", HOST)
    return LIB


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv, ptxas_info="--ptxas" in sys.argv))
