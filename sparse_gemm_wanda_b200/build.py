"""Build the CUDA library ``libpatch_b200.so`` in-tree for sm_100a.

``python -m sparse_gemm_wanda_b200.build`` (or ``build()``) compiles every
``csrc/*.cu`` with nvcc for ``compute_100a``/``sm_100a`` and links one shared
library next to this file, and ``csrc/torch_binding.cpp`` with g++ against the
installed PyTorch into ``_patch_torch.so`` beside it.  nvcc cross-compiles, so
no GPU is needed to build.
"""
from __future__ import annotations

import glob
import os
import shutil
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
OUT = os.path.join(HERE, "libpatch_b200.so")
BINDING_SRC = os.path.join(CSRC, "torch_binding.cpp")
BINDING_OUT = os.path.join(HERE, "_patch_torch.so")
BUILD_DIR = os.path.join(ROOT, "_build")

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
         "-Xptxas", "-v", "-I", INCLUDE, "-I", CSRC]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", shutil.which("nvcc")):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA library cannot be built")


def _stale(srcs, out) -> bool:
    if not os.path.exists(out):
        return True
    t = os.path.getmtime(out)
    deps = srcs + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) + \
        glob.glob(os.path.join(INCLUDE, "*.h")) + [os.path.abspath(__file__)]
    return any(os.path.getmtime(d) > t for d in deps)


def binding_target() -> str:
    """The PyTorch and Python that a binding is built against, and for."""
    import sysconfig

    import torch

    return f"torch {torch.__version__}, {sysconfig.get_config_var('SOABI')}"


def _build_binding() -> None:
    """The CPython module over PyTorch tensors (csrc/torch_binding.cpp)."""
    import sysconfig

    import torch

    target = binding_target()
    base = os.path.dirname(torch.__file__)
    include = [os.path.join(base, "include"), os.path.join(base, "include", "torch", "csrc", "api", "include"),
               os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include")]
    lib = os.path.join(base, "lib")
    tmp = BINDING_OUT + ".tmp"
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           f'-DPATCH_BUILT_FOR="{target}"', "-I", sysconfig.get_path("include"), "-I", INCLUDE, *[f"-isystem{p}" for p in include], BINDING_SRC,
           "-o", tmp, "-L", lib, f"-Wl,-rpath,{lib}", "-ltorch_python", "-ltorch_cpu", "-ltorch_cuda", "-lc10",
           "-lc10_cuda"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on {BINDING_SRC}:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, BINDING_OUT)
    with open(_binding_stamp(), "w") as fh:
        fh.write(target)


def _binding_stamp() -> str:
    return os.path.join(BUILD_DIR, "_patch_torch.txt")


def _stale_binding() -> bool:
    if not os.path.exists(BINDING_OUT) or not os.path.exists(_binding_stamp()):
        return True
    with open(_binding_stamp()) as fh:
        if fh.read() != binding_target():
            return True
    t = os.path.getmtime(BINDING_OUT)
    deps = [BINDING_SRC, os.path.join(INCLUDE, "patch.h"), os.path.abspath(__file__)]
    return any(os.path.getmtime(d) > t for d in deps)


def build(force: bool = False, verbose: bool = False) -> str:
    """Both, the CUDA library first: it needs no PyTorch."""
    os.makedirs(BUILD_DIR, exist_ok=True)
    srcs = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    if force or _stale(srcs, OUT):
        _build_library(srcs, verbose)
    if force or _stale_binding():
        _build_binding()
    return OUT


def _build_library(srcs, verbose: bool) -> None:
    cc = nvcc()

    def compile_one(src):
        obj = os.path.join(BUILD_DIR, os.path.basename(src) + ".o")
        cmd = [cc, *ARCH, *FLAGS, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        with open(obj + ".ptxas.txt", "w") as fh:
            fh.write(r.stderr)
        if verbose:
            sys.stderr.write(r.stderr)
        return obj

    with ThreadPoolExecutor(max_workers=min(8, len(srcs))) as ex:
        objs = list(ex.map(compile_one, srcs))
    tmp = OUT + ".tmp"
    cmd = [cc, *ARCH, "-shared", "-o", tmp, *objs, "-lcudart_static", "-lrt", "-ldl", "-lpthread"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, OUT)


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
