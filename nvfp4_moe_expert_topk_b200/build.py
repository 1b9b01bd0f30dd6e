"""Builds libnvfp4moe.so (the C-ABI CUDA library) in-tree for sm_100a, and
_binding.so, the Python module that checks and passes the layer operators'
tensors.

    python -m nvfp4_moe_expert_topk_b200.build [--force]
"""
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(HERE, "libnvfp4moe.so")
BINDING = os.path.join(HERE, "_binding.so")
SOURCES = ["api.cu", "api_layer.cu", "front.cu", "kernels.cu", "gemm.cu", "noalloc.cu", "ceiling.cu", "norm.cu",
           "gemv.cu", "balance.cu"]
HEADERS = ["internal.h", "ptx.cuh", "quant.cuh"]
CXX = os.environ.get("CXX", "g++")
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall",
         "--expt-relaxed-constexpr", "-I", os.path.join(ROOT, "include")]


def _newest_input():
    paths = [os.path.join(CSRC, f) for f in SOURCES + HEADERS]
    paths.append(os.path.join(ROOT, "include", "nvfp4moe.h"))
    paths.append(os.path.abspath(__file__))
    return max(os.path.getmtime(p) for p in paths)


def build_binding(force: bool = False, verbose: bool = False) -> str:
    """Compiles csrc/binding.cpp against the installed torch (host code only)."""
    import torch
    src, header = os.path.join(CSRC, "binding.cpp"), os.path.join(ROOT, "include", "nvfp4moe.h")
    stamp = BINDING + ".torch"           # the torch that the module was built against
    built_for = f"{torch.__version__} {sys.version_info[:2]}"
    newest = max(os.path.getmtime(p) for p in (src, header, os.path.abspath(__file__)))
    if not force and os.path.exists(BINDING) and os.path.getmtime(BINDING) >= newest and os.path.exists(stamp):
        with open(stamp) as f:
            if f.read() == built_for:
                return BINDING
    base = os.path.dirname(os.path.abspath(torch.__file__))
    cuda = os.path.dirname(os.path.dirname(shutil.which(NVCC) or NVCC))
    includes = [os.path.join(base, "include"), sysconfig.get_paths()["include"], os.path.join(cuda, "include"),
                os.path.join(ROOT, "include")]
    tmp = BINDING + ".tmp"
    cmd = [CXX, "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", *(f"-I{i}" for i in includes), src,
           "-o", tmp, "-L" + os.path.join(base, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda"]
    if verbose:
        print(" ".join(cmd))
    subprocess.run(cmd, check=True)
    os.replace(tmp, BINDING)
    with open(stamp, "w") as f:
        f.write(built_for)
    return BINDING


def build_library(force: bool = False, verbose: bool = False, ptxas_info: bool = False) -> str:
    """Compiles the CUDA sources (nvcc alone: neither torch nor its headers)."""
    if not force and os.path.exists(LIB) and os.path.getmtime(LIB) >= _newest_input():
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    objs = []
    for src in SOURCES:
        obj = os.path.join(BUILD, src.replace(".cu", ".o"))
        cmd = [NVCC, *ARCH, *FLAGS, "-c", os.path.join(CSRC, src), "-o", obj]
        if ptxas_info:
            cmd += ["-Xptxas", "-v"]
        if verbose:
            print(" ".join(cmd))
        subprocess.run(cmd, check=True)
        objs.append(obj)
    tmp = LIB + ".tmp"
    subprocess.run([NVCC, *ARCH, "-shared", "-o", tmp, *objs], check=True)
    os.replace(tmp, LIB)
    return LIB


def build(force: bool = False, verbose: bool = False, ptxas_info: bool = False) -> str:
    """The library, then the Python module.  Where the module cannot be built
    (no torch, no host compiler) the library is there all the same, and the
    entry points that need the module say that it is missing."""
    build_library(force, verbose, ptxas_info)
    try:
        build_binding(force, verbose)
    except (ImportError, OSError, subprocess.CalledProcessError) as e:
        for path in (BINDING, BINDING + ".torch"):       # none of older sources
            if os.path.exists(path):
                os.remove(path)
        print(f"{BINDING} was not built: {e}", file=sys.stderr)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True, ptxas_info="--ptxas-info" in sys.argv))
