"""Build the sm_100a shared library ``libsvdq.so`` in-tree with nvcc, and the
native torch calls ``_svdq_torch.so`` on top of it with the host compiler.

The library is the product: the C-ABI calls of include/svdq.h and the CUDA
kernels behind them.  It is compiled for sm_100a only (B200), and nvcc alone
builds it.  The torch calls need torch, Python's headers and g++ as well; where
one of them is missing the build says so and leaves them out.
"""

from __future__ import annotations

import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libsvdq.so")
SOURCES = [os.path.join(CSRC, "svdq.cu")]
TORCH_SOURCE = os.path.join(CSRC, "torch_calls.cpp")
TORCH_LIB = os.path.join(HERE, "_svdq_torch.so")
HEADER = os.path.join(HERE, "..", "include", "svdq.h")
DEPS = SOURCES + [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cuh")] + [
    HEADER]

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-lineinfo", "-O3", "-std=c++17",
    "-Xcompiler", "-fPIC", "-shared", "-cudart", "shared",
]


def nvcc() -> str:
    cand = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


def _stale(lib: str, deps) -> bool:
    if not os.path.exists(lib):
        return True
    t = os.path.getmtime(lib)
    return any(os.path.getmtime(d) > t for d in deps if os.path.exists(d))


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile what is missing or older than its sources; the path of libsvdq.so."""
    if force or _stale(LIB, DEPS):
        cmd = [nvcc()] + NVCC_FLAGS + (["-Xptxas", "-v"] if verbose else []) + ["-o", LIB + ".tmp"] + SOURCES
        subprocess.check_call(cmd, cwd=CSRC)
        os.replace(LIB + ".tmp", LIB)
    missing = torch_calls_missing()
    if missing:
        print(f"_svdq_torch.so not built: {missing} (libsvdq.so, the C ABI, is)", file=sys.stderr)
    elif force or _stale(TORCH_LIB, [TORCH_SOURCE, HEADER]) or not _built_for_this_torch():
        build_torch_calls()
    return LIB


def torch_calls_missing() -> str:
    """What the torch calls would need and this machine lacks ("" if nothing)."""
    try:
        import torch  # noqa: F401
    except ImportError:
        return "torch cannot be imported"
    if not os.path.exists(os.path.join(sysconfig.get_paths()["include"], "Python.h")):
        return "Python.h is missing"
    return "" if shutil.which("g++") else "g++ is missing"


def torch_tag() -> str:
    """What _svdq_torch.so is built for and holds as `built_for`: torch's C++
    interface and Python's change between versions."""
    import torch
    return f"torch {torch.__version__}, {sys.implementation.cache_tag}"


def _built_for_this_torch() -> bool:
    with open(TORCH_LIB, "rb") as f:
        return torch_tag().encode() + b"\0" in f.read()


def build_torch_calls() -> str:
    """_svdq_torch.so: torch's headers, its C++ libraries (found loaded at run
    time, after `import torch`) and libsvdq.so beside it."""
    import torch
    from torch.utils.cpp_extension import include_paths, library_paths
    inc = include_paths() + [sysconfig.get_paths()["include"], os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include")]
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}",
           f'-DSVDQ_BUILT_FOR="{torch_tag()}"']
    cmd += [f"-I{d}" for d in inc if os.path.isdir(d)]
    cmd += [TORCH_SOURCE, "-o", TORCH_LIB + ".tmp"] + [f"-L{d}" for d in library_paths()]
    cmd += ["-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_cuda", "-ltorch_python", f"-L{HERE}", "-l:libsvdq.so", "-Wl,-rpath,$ORIGIN"]
    subprocess.check_call(cmd, cwd=CSRC)
    os.replace(TORCH_LIB + ".tmp", TORCH_LIB)
    return TORCH_LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
