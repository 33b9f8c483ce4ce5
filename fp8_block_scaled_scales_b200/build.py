"""Build libdg.so (the sm_100a CUDA kernels and their C ABI) in-tree with nvcc, and
_dgtorch.so (the expert-layer calls for torch tensors, on top of that C ABI) with g++.

    python -m fp8_block_scaled_scales_b200.build [--force] [--verbose]

Output: fp8_block_scaled_scales_b200/libdg.so and _dgtorch.so.  nvcc cross-compiles
for sm_100a without a GPU.  The CUDA runtime is linked statically; the driver API is
reached through cudaGetDriverEntryPoint, so the library needs no -lcuda.
"""
from __future__ import annotations

import glob
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libdg.so")
EXT_SRC = os.path.join(CSRC, "torch_binding.cpp")
EXT = os.path.join(HERE, "_dgtorch.so")
EXT_FOR = os.path.join(HERE, "_build", "_dgtorch.for")  # the torch and Python that EXT was built against
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]


def nvcc_path() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _stale() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    deps = sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h"))
    deps.append(os.path.join(ROOT, "include", "dg.h"))
    return any(os.path.getmtime(d) > t for d in deps)


def _ext_stale(built_for: str) -> bool:
    """Whether EXT is missing, older than its sources, or built against another torch or Python."""
    if not (os.path.exists(EXT) and os.path.exists(EXT_FOR)):
        return True
    with open(EXT_FOR) as f:
        if f.read() != built_for:
            return True
    return any(os.path.getmtime(d) > os.path.getmtime(EXT) for d in (EXT_SRC, os.path.join(ROOT, "include", "dg.h")))


def _build_ext(force: bool) -> None:
    import torch
    built_for = f"torch {torch.__version__} in {os.path.dirname(torch.__file__)}, {sys.implementation.cache_tag}\n"
    if not force and not _ext_stale(built_for):
        return
    home = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc_path())))
    includes = [os.path.join(home, "include"), os.path.join(home, "include", "torch", "csrc", "api", "include"),
                os.path.join(cuda, "include")]
    tmp = EXT + ".tmp"
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           "-I", sysconfig.get_paths()["include"]]
    for path in includes:
        cmd += ["-isystem", path]
    cmd += [EXT_SRC, "-o", tmp, "-L", os.path.join(home, "lib"), "-lc10", "-lc10_cuda", "-ltorch", "-ltorch_cpu", "-ltorch_cuda",
            "-ltorch_python", "-L", HERE, "-l:libdg.so", "-Wl,-rpath,$ORIGIN"]
    subprocess.check_call(cmd)
    os.replace(tmp, EXT)
    os.makedirs(os.path.dirname(EXT_FOR), exist_ok=True)
    with open(EXT_FOR, "w") as f:
        f.write(built_for)


def build(force: bool = False, verbose: bool = False) -> str:
    _build_lib(force, verbose)
    _build_ext(force)
    return LIB


def _build_lib(force: bool, verbose: bool) -> str:
    if not force and not _stale():
        return LIB
    nvcc = nvcc_path()
    build_dir = os.path.join(HERE, "_build")
    os.makedirs(build_dir, exist_ok=True)
    common = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC,-O2",
                     "-I", os.path.join(ROOT, "include"), "--expt-relaxed-constexpr", "-rdc=false"]
    if verbose:
        common += ["-Xptxas", "-v"]
    objs = []
    for src in sources():
        obj = os.path.join(build_dir, os.path.basename(src)[:-3] + ".o")
        cmd = [nvcc] + common + ["-c", src, "-o", obj]
        subprocess.check_call(cmd)
        objs.append(obj)
    tmp = LIB + ".tmp"
    subprocess.check_call([nvcc] + ARCH + ["-shared", "-cudart", "static", "-o", tmp] + objs)
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="--verbose" in sys.argv))
