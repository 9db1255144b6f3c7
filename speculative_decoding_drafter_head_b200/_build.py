"""Build the CUDA library ``libdspark.so`` in-tree with nvcc for sm_100a, and the extension
module through which Python makes the verification pass's calls."""
from __future__ import annotations

import glob
import os
import shutil
import subprocess

PKG = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(PKG, "csrc")
ROOT = os.path.dirname(PKG)
LIB = os.path.join(PKG, "libdspark.so")

NVCC_FLAGS = [
    "-O3", "-std=c++17", "-gencode", "arch=compute_100a,code=sm_100a", "-lineinfo",
    "-Xcompiler", "-fPIC", "-shared",
]


def _nvcc() -> str:
    path = shutil.which("nvcc")
    if path:
        return path
    cand = "/usr/local/cuda/bin/nvcc"
    if os.path.exists(cand):
        return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libdspark.so")


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cuh")) +
                  glob.glob(os.path.join(CSRC, "*.h")) +
                  [os.path.join(ROOT, "include", "dspark.h")])


def _older(path, sources) -> bool:
    if not os.path.exists(path):
        return True
    t = os.path.getmtime(path)
    return any(os.path.getmtime(s) > t for s in sources)


def calls_path() -> str:
    """Where the extension module for this torch, its C++ ABI and this interpreter stands: it reads
    tensors through their inline accessors, so a file built for another must not be loaded."""
    import sysconfig

    import torch
    return os.path.join(PKG, f"_dspark_calls.torch{torch.__version__}"
                             f"-abi{int(torch._C._GLIBCXX_USE_CXX11_ABI)}"
                             f"{sysconfig.get_config_var('EXT_SUFFIX')}")


def _calls_sources():
    return [os.path.join(CSRC, "binding.cpp"), os.path.join(ROOT, "include", "dspark.h")]


def stale() -> bool:
    return _older(LIB, _sources())


def calls_stale() -> bool:
    return _older(calls_path(), _calls_sources())


def build_calls(force: bool = False, verbose: bool = False) -> str:
    """Compile csrc/binding.cpp against this interpreter and its torch."""
    path = calls_path()
    if not force and not calls_stale():
        return path
    import sysconfig

    import torch
    from torch.utils import cpp_extension
    tmp = path + f".tmp{os.getpid()}"
    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    cuda = os.path.dirname(os.path.dirname(_nvcc()))
    include = [*cpp_extension.include_paths(), os.path.join(cuda, "include"),
               sysconfig.get_paths()["include"]]
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           *[f"-isystem{i}" for i in include], "-o", tmp, os.path.join(CSRC, "binding.cpp"),
           f"-L{lib}", "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch", "-ltorch_python"]
    if verbose:
        print(" ".join(cmd))
    subprocess.check_call(cmd)
    os.replace(tmp, path)
    return path


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile csrc/dspark_api.cu (which includes every kernel) into libdspark.so."""
    if not force and not stale():
        return LIB
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [_nvcc(), *NVCC_FLAGS, "-I", os.path.join(ROOT, "include"), "-o", tmp,
           os.path.join(CSRC, "dspark_api.cu")]
    if verbose:
        print(" ".join(cmd))
    subprocess.check_call(cmd)
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force=True, verbose=True))
    print(build_calls(force=True, verbose=True))
