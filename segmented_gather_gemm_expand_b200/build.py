"""Build libsgmv.so (the C-ABI CUDA library) in-tree for sm_100a, and the
CPython extension that marshals torch tensors for its large products.

Usage: python segmented_gather_gemm_expand_b200/build.py [--force]
(run as a script: importing the package needs the library this builds)
"""
import glob
import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(HERE, "libsgmv.so")
BINDING = os.path.join(HERE, "_binding.so")
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")

FLAGS = ["-gencode", "arch=compute_100a,code=sm_100a", "-lineinfo", "-O3", "-std=c++17",
         "--expt-relaxed-constexpr", "-Xcompiler", "-fPIC,-fvisibility=hidden", "-shared",
         "-Xptxas", "-v", "-I", INCLUDE, "-I", CSRC]


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cuh")) +
                  [os.path.join(INCLUDE, "sgmv.h")])


def binding_target() -> str:
    """The Python and torch that the extension is compiled for; it holds this text as `built_for`."""
    import torch
    return f"python {sys.version_info.major}.{sys.version_info.minor}, torch {torch.__version__}"


def binding_is_current() -> bool:
    if not os.path.exists(BINDING):
        return False
    if os.path.getmtime(BINDING) < max(os.path.getmtime(s) for s in (os.path.join(CSRC, "binding.cpp"),
                                                                     os.path.join(INCLUDE, "sgmv.h"))):
        return False
    with open(BINDING, "rb") as f:
        return binding_target().encode() + b"\0" in f.read()


def build_binding(force: bool = False) -> str:
    src = os.path.join(CSRC, "binding.cpp")
    if not force and binding_is_current():
        return BINDING
    import sysconfig

    import torch
    root = os.path.dirname(torch.__file__)
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-shared", "-fPIC", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", f'-DBUILT_FOR="{binding_target()}"',
           "-I", INCLUDE,
           "-isystem", os.path.join(root, "include"),
           "-isystem", os.path.join(root, "include", "torch", "csrc", "api", "include"),
           "-isystem", sysconfig.get_paths()["include"], "-isystem", "/usr/local/cuda/include",
           "-o", BINDING + ".tmp", src, "-L", os.path.join(root, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10_cuda",
           "-lc10"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        sys.stderr.write(r.stdout + r.stderr)
        raise RuntimeError("the compiler failed building _binding.so")
    os.replace(BINDING + ".tmp", BINDING)
    return BINDING


def build(force: bool = False, verbose: bool = False) -> str:
    build_binding(force)
    if not force and os.path.exists(LIB):
        newest = max(os.path.getmtime(s) for s in sources())
        if os.path.getmtime(LIB) >= newest:
            return LIB
    cmd = [NVCC, *FLAGS, "-o", LIB + ".tmp", os.path.join(CSRC, "sgmv.cu")]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        sys.stderr.write(r.stdout + r.stderr)
        raise RuntimeError("nvcc failed building libsgmv.so")
    if verbose:
        sys.stderr.write(r.stderr)
    os.replace(LIB + ".tmp", LIB)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))
