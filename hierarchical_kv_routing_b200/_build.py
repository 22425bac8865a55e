"""Build libhga.so in-tree: every csrc/*.cu compiled for sm_100a with nvcc,
objects under _build/, linked into hierarchical_kv_routing_b200/libhga.so; and
_paged.so, the compiled part of the Python binding (csrc/binding.cpp, host code
against the installed torch and libhga.so)."""
from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import subprocess
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libhga.so")
EXT = os.path.join(PKG, "_paged.so")
EXT_SRC = os.path.join(CSRC, "binding.cpp")
INCLUDE = os.path.join(os.path.dirname(PKG), "include")

NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-I", INCLUDE,
         "--expt-relaxed-constexpr"]


def _deps_mtime() -> float:
    files = glob.glob(os.path.join(CSRC, "*.cu*")) + glob.glob(os.path.join(INCLUDE, "*.h"))
    return max(os.path.getmtime(f) for f in files)


def _compile(src: str) -> str:
    obj = os.path.join(BUILD, os.path.basename(src) + ".o")
    if os.path.exists(obj) and os.path.getmtime(obj) >= _deps_mtime():
        return obj
    cmd = [NVCC, *ARCH, *FLAGS, "-c", src, "-o", obj + ".tmp"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
    os.replace(obj + ".tmp", obj)
    return obj


def _build_ext(force: bool) -> None:
    """binding.cpp -> _paged.so (after libhga.so, which it links)."""
    newest = max(os.path.getmtime(f) for f in [EXT_SRC, *glob.glob(os.path.join(INCLUDE, "*.h"))])
    if not force and os.path.exists(EXT) and os.path.getmtime(EXT) >= newest:
        return
    import torch
    from torch.utils import cpp_extension
    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    cuda = os.path.join(os.path.dirname(os.path.dirname(NVCC)), "include")
    inc = [f"-I{p}" for p in [*cpp_extension.include_paths(), cuda, INCLUDE,
                              sysconfig.get_paths()["include"]]]
    tmp = EXT + f".tmp{os.getpid()}"
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-w", *inc, EXT_SRC, "-o", tmp,
           f"-L{lib}", "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10", "-lc10_cuda", f"-L{PKG}",
           "-lhga", "-Wl,-rpath,$ORIGIN", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed for {EXT_SRC}:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, EXT)


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile (incrementally) and link; returns the library path."""
    _build_lib(force, verbose)
    _build_ext(force)
    return LIB


def _build_lib(force: bool, verbose: bool) -> str:
    os.makedirs(BUILD, exist_ok=True)
    if not force and os.path.exists(LIB) and os.path.getmtime(LIB) >= _deps_mtime():
        return LIB
    srcs = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    if force:
        for o in glob.glob(os.path.join(BUILD, "*.o")):
            os.remove(o)
    with cf.ThreadPoolExecutor(max_workers=min(8, len(srcs))) as ex:
        objs = list(ex.map(_compile, srcs))
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [NVCC, *ARCH, "-shared", "-Xcompiler", "-fPIC", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    if verbose:
        print("built", LIB)
    return LIB


if __name__ == "__main__":
    build(verbose=True)
