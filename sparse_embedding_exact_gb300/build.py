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
from typing import Optional

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


def _newer(target, inputs) -> bool:
    """Whether `target` exists and no input changed after it was made."""
    return os.path.exists(target) and all(os.path.getmtime(f) <= os.path.getmtime(target) for f in inputs)


def _library_up_to_date() -> bool:
    return _newer(LIB, sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(INCLUDE, "*.h")))


def _torch() -> str:
    import torch

    return str(torch.__version__)


def binding_torch() -> Optional[str]:
    """The version of torch that the binding was built against (its C++
    interface changes between versions); None: there is no binding."""
    try:
        with open(BINDING + ".torch") as f:
            return f.read() if os.path.exists(BINDING) else None
    except OSError:
        return None


def _binding_up_to_date() -> bool:
    return binding_torch() == _torch() and _newer(BINDING, [_binding_source()] + glob.glob(os.path.join(INCLUDE, "*.h")))


def up_to_date() -> bool:
    return _library_up_to_date() and _binding_up_to_date()


def _run(cmd, what: str, verbose: bool = False):
    if verbose:
        print(" ".join(cmd), file=sys.stderr)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{what}:\n{r.stdout}\n{r.stderr}")
    if verbose and (r.stdout or r.stderr):
        print(r.stdout + r.stderr, file=sys.stderr)


def _link(target: str, cmd, what: str):
    """Runs a link command, whose output replaces `target` once it is whole."""
    tmp = f"{target}.{os.getpid()}.tmp"
    _run([cmd[0], "-shared", "-o", tmp] + cmd[1:], what)
    os.replace(tmp, target)


def _compile_binding():
    """(object, torch's library folders) of the binding."""
    import sysconfig

    import torch
    from torch.utils import cpp_extension

    obj = os.path.join(BUILD, "binding.o")
    include = [INCLUDE, CSRC, sysconfig.get_paths()["include"]] + cpp_extension.include_paths("cuda")
    abi = int(torch._C._GLIBCXX_USE_CXX11_ABI)
    _run([shutil.which("g++") or "g++", "-c", _binding_source(), "-o", obj, "-O2", "-std=c++17", "-fPIC",
          "-fvisibility=hidden", f"-D_GLIBCXX_USE_CXX11_ABI={abi}"] + ["-I" + i for i in include],
         f"g++ failed on {_binding_source()}")
    return obj, cpp_extension.library_paths("cuda")


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    """Builds what is not up to date.  The library needs nvcc alone and is
    there also where the binding, which needs torch's C++ headers, fails; that
    is raised afterwards."""
    library, binding = force or not _library_up_to_date(), force or not _binding_up_to_date()
    if not (library or binding):
        return LIB
    os.makedirs(BUILD, exist_ok=True)

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
        _run([nvcc(), "-c", src, "-o", obj] + ARCH + NVCC_FLAGS + list(extra_flags), f"nvcc failed on {src}", verbose)
        return obj

    with ThreadPoolExecutor(max_workers=max(1, min(16, len(sources()) + 1))) as ex:
        compiled = ex.submit(_compile_binding) if binding else None
        if library:
            objs = list(ex.map(compile_one, sources()))
            _link(LIB, [nvcc()] + objs + ARCH + ["-cudart", "static", "-Xcompiler", "-fPIC"], "nvcc link failed")
    if binding:
        obj, torch_libs = compiled.result()
        cmd = [shutil.which("g++") or "g++", obj, "-L" + BUILD, "-lsparsecos", "-Wl,-rpath,$ORIGIN"]
        for d in torch_libs:
            cmd += ["-L" + d, "-Wl,-rpath," + d]
        _link(BINDING, cmd + ["-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10", "-lc10_cuda"], f"linking {BINDING} failed")
        with open(BINDING + ".torch", "w") as f:
            f.write(_torch())
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))
