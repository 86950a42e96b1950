"""Builds libbitnet_b200.so in-tree with nvcc for sm_100a (B200).

The CUDA runtime is linked statically and the driver API is reached through
cudaGetDriverEntryPoint, so the library loads on a machine without a GPU
driver (where every compute call then returns BITNET_ERR_CUDA).  Beside it the
native binding of the 4-bit functions (_binding.so, g++ against the installed
torch; left out where there is none).
"""
from __future__ import annotations

import glob
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libbitnet_b200.so")
BINDING = os.path.join(PKG, "_binding.so")
BINDING_SRC = os.path.join(CSRC, "binding.cpp")

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-lineinfo", "-std=c++17",
    "--expt-relaxed-constexpr",
    "-Xcompiler", "-fPIC,-fvisibility=hidden",
    "-shared", "--cudart", "static",
]


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cuh"))
                  + glob.glob(os.path.join(CSRC, "*.h")) + [os.path.join(INCLUDE, "bitnet_b200.h")])


def newer(target, inputs) -> bool:
    """Whether `target` is there and none of `inputs` is younger."""
    if not os.path.exists(target):
        return False
    t = os.path.getmtime(target)
    return all(os.path.getmtime(s) <= t for s in inputs)


def up_to_date() -> bool:
    return newer(LIB, sources())


def build_binding(force: bool = False, verbose: bool = False):
    """Builds the binding; without torch there is nothing to bind to, and the C library is complete by itself."""
    try:
        import torch
    except ImportError:
        torch = None
    if torch is None or torch.version.cuda is None:
        print("torch is not installed, or without CUDA: the native binding of the 4-bit functions is not built",
              file=sys.stderr)
        return None
    # a binding fits one torch and one Python: which ones it was built for stands beside it
    stamp, fits = BINDING[:-len(".so")] + ".stamp", f"{torch.__version__} {sys.implementation.cache_tag}"
    if not force and newer(BINDING, [BINDING_SRC, os.path.join(INCLUDE, "bitnet_b200.h")]) and os.path.exists(stamp):
        with open(stamp, encoding="utf-8") as f:
            if f.read() == fits:
                return BINDING
    tdir = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"))
    includes = [INCLUDE, os.path.join(tdir, "include"), os.path.join(tdir, "include", "torch", "csrc", "api", "include"),
                sysconfig.get_paths()["include"], os.path.join(cuda, "include")]
    cmd = ["g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-fvisibility=hidden",
           f'-DBINDING_TORCH="{torch.__version__}"',
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}", *(f"-I{i}" for i in includes),
           BINDING_SRC, "-o", BINDING + ".tmp", f"-L{os.path.join(tdir, 'lib')}", "-ltorch_python", "-ltorch",
           "-ltorch_cpu", "-ltorch_cuda", "-lc10", "-lc10_cuda", f"-L{PKG}", "-l:libbitnet_b200.so", "-Wl,-rpath,$ORIGIN"]
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.run(cmd, check=True)
    os.replace(BINDING + ".tmp", BINDING)
    with open(stamp, "w", encoding="utf-8") as f:
        f.write(fits)
    return BINDING


def build(force: bool = False, verbose: bool = False, extra=None) -> str:
    if force or not up_to_date():
        cmd = ["nvcc", *NVCC_FLAGS, *(extra or []), "-I", INCLUDE,
               "-o", LIB + ".tmp", os.path.join(CSRC, "bitnet_b200.cu")]
        if verbose:
            print(" ".join(cmd), flush=True)
        subprocess.run(cmd, check=True)
        os.replace(LIB + ".tmp", LIB)
    build_binding(force, verbose)
    return LIB


if __name__ == "__main__":
    extra = ["-Xptxas", "-v"] if "--ptxas-v" in sys.argv else None
    print(build(force="--force" in sys.argv or extra is not None, verbose=True, extra=extra))
