"""Build ``libmoe_mxfp4.so`` in-tree with nvcc for sm_100a (runs without a GPU)."""
from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libmoe_mxfp4.so")
# The same library with the layer's and the tiled products' stores at computed offsets checked against
# their buffers (-DMOE_DEBUG_BOUNDS): an out-of-range store is skipped and MOE_ERR_BOUNDS recorded.
LIB_BOUNDS = os.path.join(PKG, "libmoe_mxfp4_bounds.so")
# The tensor-argument part of the binding (compiled against this torch and Python, named by them).
MARSHAL_SRC = os.path.join(PKG, "binding", "marshal.cpp")
BUILD_DIR = os.path.join(PKG, "_build")

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
    "-I", INCLUDE, "-I", CSRC,
]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def dependencies():
    return sources() + [f for d, p in ((CSRC, "*.cuh"), (CSRC, "*.h"), (INCLUDE, "*.h")) for f in glob.glob(os.path.join(d, p))]


def _deps_mtime() -> float:
    return max(os.path.getmtime(f) for f in dependencies())


def up_to_date(lib: str = LIB) -> bool:
    return os.path.exists(lib) and os.path.getmtime(lib) >= _deps_mtime()


def build_marshal(force: bool = False) -> str:
    """Compile the binding's part in C++ with the host compiler."""
    from mxfp4_expert_gemm_b200 import marshal_path
    lib = marshal_path()
    newest = max(os.path.getmtime(f) for f in (MARSHAL_SRC, os.path.join(INCLUDE, "moe_mxfp4.h")))
    if not force and os.path.exists(lib) and os.path.getmtime(lib) >= newest:
        return lib
    import sysconfig

    import torch
    root = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(_nvcc()))
    tmp = lib + f".tmp{os.getpid()}"
    cmd = ["g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-Wno-deprecated-declarations", MARSHAL_SRC, "-o", tmp,
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", "-I", INCLUDE,
           "-I", os.path.join(root, "include"), "-I", os.path.join(root, "include", "torch", "csrc", "api", "include"),
           "-I", sysconfig.get_paths()["include"], "-I", os.path.join(cuda, "include"),
           "-L", os.path.join(root, "lib"), "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10", "-lc10_cuda"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed for {MARSHAL_SRC}:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, lib)
    return lib


def build(force: bool = False, verbose: bool = False, extra_flags=(), bounds: bool = False) -> str:
    """Compile the library (with bounds=True: the bounds-checking build, LIB_BOUNDS)."""
    lib = LIB_BOUNDS if bounds else LIB
    build_marshal(force and not bounds)
    if bounds:
        extra_flags = (*extra_flags, "-DMOE_DEBUG_BOUNDS")
    if not force and up_to_date(lib):
        return lib
    nvcc = _nvcc()
    build_dir = os.path.join(BUILD_DIR, "bounds" if bounds else "release")
    os.makedirs(build_dir, exist_ok=True)
    objs = []

    def compile_one(src):
        obj = os.path.join(build_dir, os.path.basename(src) + ".o")
        cmd = [nvcc, *NVCC_FLAGS, *extra_flags, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            print(r.stdout, r.stderr, file=sys.stderr)
        return obj

    with cf.ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 1)) as ex:
        objs = list(ex.map(compile_one, sources()))
    tmp = lib + f".tmp{os.getpid()}"
    cmd = [nvcc, "-shared", "-gencode", "arch=compute_100a,code=sm_100a", *objs, "-o", tmp]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, lib)
    return lib


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True, bounds="--bounds" in sys.argv))
