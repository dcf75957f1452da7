"""Build the CUDA library (sm_100a) in-tree: group_quantized_w4a4_b200/_lib/libapex_w4a4.so,
and the torch side of its newer calls, _lib/apex_torch-<versions of torch and Python>.so (plain
C++ against torch's headers, whose ABI changes with both).

    python -m group_quantized_w4a4_b200.build [--force]

nvcc cross-compiles for sm_100a without a GPU; the result is a plain shared library with
the C ABI of include/apex_w4a4.h (static CUDA runtime; the driver's tensor-map encoder is
looked up at run time, so there is no link-time dependency on libcuda).
"""
from __future__ import annotations

import glob
import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB_DIR = os.path.join(PKG, "_lib")
LIB_PATH = os.path.join(LIB_DIR, "libapex_w4a4.so")
TORCH_SRC = os.path.join(CSRC, "torch_binding.cpp")
ARCH_FLAGS = ["-gencode", "arch=compute_100a,code=sm_100a"]


def _nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build the library")


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cuh"))
                  + glob.glob(os.path.join(INCLUDE, "*.h")))


def is_stale() -> bool:
    if not os.path.exists(LIB_PATH):
        return True
    t = os.path.getmtime(LIB_PATH)
    return any(os.path.getmtime(s) > t for s in _sources())


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile the library if a source is newer than it (or `force`); return its path."""
    if not force and not is_stale():
        return LIB_PATH
    os.makedirs(LIB_DIR, exist_ok=True)
    tmp = LIB_PATH + f".tmp{os.getpid()}"
    cmd = [_nvcc(), *ARCH_FLAGS, "-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
           "-shared", f"-I{INCLUDE}", f"-I{CSRC}", "-o", tmp,
           os.path.join(CSRC, "apex_w4a4.cu")]
    if verbose:
        cmd.insert(1, "-Xptxas=-v")
    subprocess.run(cmd, check=True)
    os.replace(tmp, LIB_PATH)
    return LIB_PATH


def torch_lib_path() -> str:
    """The torch binding's file: a name for each torch and Python, so that none loads another's."""
    import torch
    version = "".join(c if c.isalnum() or c == "." else "_" for c in torch.__version__)
    return os.path.join(LIB_DIR, f"apex_torch-{version}-{sys.implementation.cache_tag}.so")


def torch_is_stale() -> bool:
    path = torch_lib_path()
    if not os.path.exists(path):
        return True
    t = os.path.getmtime(path)
    headers = glob.glob(os.path.join(INCLUDE, "*.h"))
    return any(os.path.getmtime(s) > t for s in [TORCH_SRC, *headers])


def build_torch(force: bool = False) -> str:
    """Compile the torch binding if there is none for this torch and Python, or it is older than its
    sources (or `force`); return its path."""
    path = torch_lib_path()
    if not force and not torch_is_stale():
        return path
    import sysconfig

    import torch
    from torch.utils import cpp_extension
    os.makedirs(LIB_DIR, exist_ok=True)
    tmp = path + f".tmp{os.getpid()}"
    include = [INCLUDE, sysconfig.get_paths()["include"], *cpp_extension.include_paths("cuda")]
    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    cxx = shutil.which("g++") or "g++"
    subprocess.run([cxx, "-O2", "-std=c++17", "-fPIC", "-shared",
                    f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
                    *(f for i in include for f in ("-isystem", i)), TORCH_SRC, "-o", tmp,
                    f"-L{lib}", f"-Wl,-rpath,{lib}", "-ltorch_python", "-ltorch", "-ltorch_cpu",
                    "-lc10", "-lc10_cuda"], check=True)
    os.replace(tmp, path)
    return path


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
    print(build_torch(force="--force" in sys.argv))
