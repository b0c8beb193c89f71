"""Compiles the CUDA library (libsparsecos.so) for sm_103a, in-tree.

Each .cu file compiles to an object in parallel with nvcc, then nvcc links
them into one shared library with the CUDA runtime linked statically.  Beside
it, the dense operators' binding to torch tensors (_dense_binding.so, a Python
module that calls the library) compiles with the host compiler.
"""
from __future__ import annotations

import glob
import os
import shutil
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(BUILD, "libsparsecos.so")
BINDING = os.path.join(BUILD, "_dense_binding.so")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall",
              "--expt-relaxed-constexpr", f"-I{INCLUDE}", f"-I{CSRC}"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA library cannot be built")


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _binding_source():
    return os.path.join(CSRC, "binding.cpp")


def _inputs():
    return sources() + [_binding_source()] + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(INCLUDE, "*.h"))


def up_to_date() -> bool:
    if not os.path.exists(LIB) or not os.path.exists(BINDING):
        return False
    t = min(os.path.getmtime(LIB), os.path.getmtime(BINDING))
    return all(os.path.getmtime(f) <= t for f in _inputs())


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    if not force and up_to_date():
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    cc = nvcc()
    objs = []

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
        cmd = [cc, "-c", src, "-o", obj] + ARCH + NVCC_FLAGS + list(extra_flags)
        if verbose:
            print(" ".join(cmd), file=sys.stderr)
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            print(r.stdout + r.stderr, file=sys.stderr)
        return obj

    def compile_binding():
        import sysconfig

        import torch
        from torch.utils import cpp_extension

        obj = os.path.join(BUILD, "binding.o")
        include = [INCLUDE, CSRC, sysconfig.get_paths()["include"]] + cpp_extension.include_paths("cuda")
        abi = int(torch._C._GLIBCXX_USE_CXX11_ABI)
        cmd = [shutil.which("g++") or "g++", "-c", _binding_source(), "-o", obj, "-O2", "-std=c++17", "-fPIC",
               "-fvisibility=hidden", f"-D_GLIBCXX_USE_CXX11_ABI={abi}"] + ["-I" + i for i in include]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"g++ failed on {_binding_source()}:\n{r.stdout}\n{r.stderr}")
        return obj, cpp_extension.library_paths("cuda")

    with ThreadPoolExecutor(max_workers=max(1, min(16, len(sources()) + 1))) as ex:
        binding = ex.submit(compile_binding)
        objs = list(ex.map(compile_one, sources()))
        binding_obj, torch_libs = binding.result()
    tmp = f"{LIB}.{os.getpid()}.tmp"
    cmd = [cc, "-shared", "-o", tmp] + objs + ARCH + ["-cudart", "static", "-Xcompiler", "-fPIC"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    tmp = f"{BINDING}.{os.getpid()}.tmp"
    cmd = [shutil.which("g++") or "g++", "-shared", "-o", tmp, binding_obj, "-L" + BUILD, "-lsparsecos", "-Wl,-rpath,$ORIGIN"]
    for d in torch_libs:
        cmd += ["-L" + d, "-Wl,-rpath," + d]
    cmd += ["-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10", "-lc10_cuda"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"linking {BINDING} failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, BINDING)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))
