"""Build liblora_sgmv.so in-tree with nvcc for sm_100a, then the binding's native
marshalling (_native-*.so) against the installed torch.  The library needs nvcc only:
without torch, or with one without CUDA, the second step is left out.

    python -m adapter_gemv_sgmv_b200.build [--force]

cudart is linked statically, so the library loads on a machine without a
GPU (its symbols can be inspected there); it needs the NVIDIA driver only
when a call reaches the device.
"""
from __future__ import annotations

import glob
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "liblora_sgmv.so")
EXT_SOURCE = os.path.join(CSRC, "binding.cpp")
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]


def nvcc() -> str:
    for c in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", shutil.which("nvcc")):
        if c and os.path.exists(c):
            return c
    raise RuntimeError("nvcc not found")


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _inputs():
    return sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(INCLUDE, "*.h"))


def stale() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    return any(os.path.getmtime(f) > t for f in _inputs())


def native_path() -> str:
    """The native module of this interpreter and torch: another one of either has its own file."""
    import torch
    tag = f"{sysconfig.get_config_var('SOABI')}-torch{torch.__version__}-abi{int(torch._C._GLIBCXX_USE_CXX11_ABI)}"
    return os.path.join(PKG, f"_native-{tag}.so")


def build_native(force: bool = False, verbose: bool = False) -> str:
    """The native half of the Python binding (host code only; needs torch with CUDA)."""
    ext = native_path()
    if not force and os.path.exists(ext) and all(
            os.path.getmtime(f) <= os.path.getmtime(ext)
            for f in [EXT_SOURCE, os.path.join(INCLUDE, "lora_sgmv.h"), os.path.abspath(__file__)]):
        return ext
    import torch
    from torch.utils import cpp_extension as ce
    cuda = os.path.dirname(os.path.dirname(nvcc()))
    inc = [INCLUDE, sysconfig.get_paths()["include"], *ce.include_paths(), os.path.join(cuda, "include")]
    lib = [*ce.library_paths(), os.path.join(cuda, "lib64")]
    tmp = ext + f".tmp{os.getpid()}"
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-shared", "-fPIC", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           *[f"-isystem{i}" for i in inc[1:]], "-I", inc[0], EXT_SOURCE, *[f"-L{d}" for d in lib],
           "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda", "-lcudart", f"-Wl,-rpath,{ce.library_paths()[0]}",
           "-o", tmp]
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.check_call(cmd)
    os.replace(tmp, ext)
    return ext


def build_library(force: bool = False, verbose: bool = False, extra=()) -> str:
    if not force and not stale():
        return LIB
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [nvcc(), *ARCH, "-lineinfo", "-O3", "-std=c++17", "-shared", "-Xcompiler", "-fPIC",
           "-Xcompiler", "-fvisibility=hidden", "--expt-relaxed-constexpr",
           "-I", INCLUDE, "-I", CSRC, *extra, *sources(), "-o", tmp]
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.check_call(cmd)
    os.replace(tmp, LIB)
    return LIB


def torch_with_cuda() -> bool:
    if importlib.util.find_spec("torch") is None:
        return False
    import torch
    return torch.version.cuda is not None


def build(force: bool = False, verbose: bool = False, extra=()) -> str:
    """The library, then (with torch) the native module, whose failure leaves the library made."""
    build_library(force, verbose, extra)
    if torch_with_cuda():
        build_native(force, verbose)
    elif verbose:
        print("no torch with CUDA: the library alone (the Python binding's native module is left out)", flush=True)
    return LIB


if __name__ == "__main__":
    force = "--force" in sys.argv
    v = "-v" in sys.argv
    extra = ["-Xptxas", "-v"] if "--ptxas" in sys.argv else []
    print(build(force=force or bool(extra), verbose=v, extra=extra))
