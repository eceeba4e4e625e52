"""Build libgqa_decode.so in-tree with nvcc for sm_103a (GB300)."""
from __future__ import annotations

import glob
import hashlib
import os
import subprocess

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
LIB_PATH = os.path.join(PKG, "libgqa_decode.so")
INCLUDE = os.path.join(ROOT, "include")
# translation units, compiled side by side
SRCS = [os.path.join(PKG, "csrc", name) for name in ("gqa_decode.cu", "fp4_decode.cu", "cache_io.cu", "prefill.cu",
                                                   "serving.cu")]

NVCC_FLAGS = ["-gencode", "arch=compute_103a,code=sm_103a", "-O3", "-lineinfo", "-std=c++17",
              "-Xcompiler", "-fPIC", "-shared", "-t", "0"]


def _sources():
    return (glob.glob(os.path.join(PKG, "csrc", "**", "*.cuh"), recursive=True)
            + glob.glob(os.path.join(PKG, "csrc", "**", "*.cu"), recursive=True)
            + glob.glob(os.path.join(PKG, "csrc", "**", "*.h"), recursive=True)
            + glob.glob(os.path.join(INCLUDE, "*.h")))


def interface() -> str:
    """A token that names the C interface: the header's digest.  The library and the
    native binding are both built with it, and the binding only calls a library of
    the same one."""
    with open(os.path.join(INCLUDE, "gqa_decode.h"), "rb") as f:
        return "h" + hashlib.sha256(f.read()).hexdigest()[:16]


def nvcc() -> str:
    cand = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile the library if it is missing or older than any source."""
    if not force and os.path.exists(LIB_PATH):
        newest = max(os.path.getmtime(s) for s in _sources())
        if os.path.getmtime(LIB_PATH) >= newest:
            return LIB_PATH
    tmp = LIB_PATH + f".tmp{os.getpid()}"
    cmd = [nvcc(), *NVCC_FLAGS, "-DGQA_INTERFACE=" + interface(), "-I" + INCLUDE, "-o", tmp, *SRCS]
    if verbose:
        print(" ".join(cmd))
    subprocess.run(cmd, check=True)
    os.replace(tmp, LIB_PATH)
    return LIB_PATH


CHECKED_LIB_PATH = os.path.join(PKG, "libgqa_decode_checked.so")


def build_checked(force: bool = False, verbose: bool = False) -> str:
    """The same library with the kernels' accesses range-checked (-DGQA_CHECKED):
    an access outside its buffer sets GQA_FLAG_BOUNDS and is redirected inside
    it.  For tests only; the product library is built without the checks."""
    if not force and os.path.exists(CHECKED_LIB_PATH):
        newest = max(os.path.getmtime(s) for s in _sources())
        if os.path.getmtime(CHECKED_LIB_PATH) >= newest:
            return CHECKED_LIB_PATH
    tmp = CHECKED_LIB_PATH + f".tmp{os.getpid()}"
    cmd = [nvcc(), *NVCC_FLAGS, "-DGQA_CHECKED", "-DGQA_INTERFACE=" + interface(), "-I" + INCLUDE, "-o", tmp, *SRCS]
    if verbose:
        print(" ".join(cmd))
    subprocess.run(cmd, check=True)
    os.replace(tmp, CHECKED_LIB_PATH)
    return CHECKED_LIB_PATH


NATIVE_SRC = os.path.join(PKG, "csrc", "binding.cpp")
NATIVE_PATH = os.path.join(PKG, "_native.so")


def native_built_for() -> str:
    """What the binding is built for, as it is written into it: torch, Python and the C interface."""
    import sysconfig

    import torch

    return f"gqa binding for torch {torch.__version__}, {sysconfig.get_config_var('SOABI')}, {interface()}"


def native_is_current(path: str) -> bool:
    """The binding is there, no older than its source and built for what runs here."""
    if not os.path.exists(path) or os.path.getmtime(path) < os.path.getmtime(NATIVE_SRC):
        return False
    with open(path, "rb") as f:
        return native_built_for().encode() in f.read()


def build_native(force: bool = False, verbose: bool = False) -> str:
    """The native binding of the cache write and read-back calls and of decode calls
    (a CPython extension against the installed torch's headers, compiled with g++)."""
    import sysconfig

    import torch

    if not force and native_is_current(NATIVE_PATH):
        return NATIVE_PATH
    cuda = os.path.dirname(os.path.dirname(nvcc()))
    home = os.path.dirname(torch.__file__)
    lib = os.path.join(home, "lib")
    includes = [INCLUDE, os.path.join(home, "include"), sysconfig.get_paths()["include"], os.path.join(cuda, "include")]
    tmp = NATIVE_PATH + f".tmp{os.getpid()}"
    cmd = ["g++", "-O2", "-std=c++17", "-shared", "-fPIC", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}",
           f'-DGQA_TORCH_VERSION="{torch.__version__}"', f'-DGQA_INTERFACE="{interface()}"',
           f'-DGQA_BUILT_FOR="{native_built_for()}"', *("-I" + i for i in includes), NATIVE_SRC, "-o", tmp, "-L" + lib,
           "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10", "-lc10_cuda"]
    if verbose:
        print(" ".join(cmd))
    subprocess.run(cmd, check=True)
    os.replace(tmp, NATIVE_PATH)
    return NATIVE_PATH
