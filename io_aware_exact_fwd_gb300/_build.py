"""Builds libfa.so in-tree with nvcc for sm_103a (no CMake, no torch extension machinery).

Each ``csrc/*.cu`` translation unit compiles in parallel; the objects link into
``io_aware_exact_fwd_gb300/lib/libfa.so`` with the CUDA runtime linked statically,
so the library needs nothing at run time but the NVIDIA driver.  ``csrc/fa_torch.cpp``,
the binding to PyTorch tensors of the calls whose host time counts, becomes
``lib/_fa_torch.so`` beside it, against the PyTorch that is installed.
"""

from __future__ import annotations

import concurrent.futures as cf
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
LIBDIR = os.path.join(PKG, "lib")
LIB = os.path.join(LIBDIR, "libfa.so")
TORCH_SRC = os.path.join(CSRC, "fa_torch.cpp")
TORCH_LIB = os.path.join(LIBDIR, "_fa_torch.so")
OBJDIR = os.path.join(ROOT, "_build", "obj")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
CFLAGS = ARCH + [
    "-O3", "-lineinfo", "-std=c++17", "--expt-relaxed-constexpr",
    "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
    "-I", INCLUDE, "-I", CSRC,
]


def _nvcc() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found")
    return cand


def _compile(src: str, extra: list[str], verbose: bool) -> str:
    obj = os.path.join(OBJDIR, os.path.basename(src) + ".o")
    cmd = [_nvcc(), *CFLAGS, *extra, "-c", src, "-o", obj]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
    if verbose and (r.stdout or r.stderr):
        print(r.stdout + r.stderr, flush=True)
    return obj


def _run(cmd: list[str], what: str):
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{what} failed:\n{r.stdout}\n{r.stderr}")


def _torch_dir() -> str:
    spec = importlib.util.find_spec("torch")  # its folder, without importing it
    if spec is None or not spec.submodule_search_locations:
        raise RuntimeError("PyTorch not found")
    return list(spec.submodule_search_locations)[0]


def _compile_torch(verbose: bool) -> str:
    obj = os.path.join(OBJDIR, "fa_torch.cpp.o")
    inc = os.path.join(_torch_dir(), "include")
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(_nvcc()))), "include")
    if not os.path.exists(os.path.join(cuda, "cuda_runtime_api.h")):
        cuda = "/usr/local/cuda/include"
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", "-isystem", inc, "-isystem",
           os.path.join(inc, "torch", "csrc", "api", "include"), "-isystem", sysconfig.get_paths()["include"], "-isystem",
           cuda, "-I", INCLUDE, "-c", TORCH_SRC, "-o", obj]
    if verbose:
        print(" ".join(cmd), flush=True)
    _run(cmd, f"g++ for {TORCH_SRC}")
    return obj


def build(verbose: bool = False, ptxas_info: bool = False) -> str:
    """Compile every kernel TU and link libfa.so and the binding.  Returns the library path."""
    os.makedirs(OBJDIR, exist_ok=True)
    os.makedirs(LIBDIR, exist_ok=True)
    sources = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    extra = ["-Xptxas", "-v"] if ptxas_info else []
    workers = min(len(sources) + 1, os.cpu_count() or 4)
    with cf.ThreadPoolExecutor(max_workers=workers) as ex:
        torch_obj = ex.submit(_compile_torch, verbose or ptxas_info)
        objs = list(ex.map(lambda s: _compile(s, extra, verbose or ptxas_info), sources))
        torch_obj = torch_obj.result()
    tmp = LIB + ".tmp"
    _run([_nvcc(), *ARCH, "-shared", "-o", tmp, *objs, "-cudart", "static"], "link of libfa.so")
    os.replace(tmp, LIB)
    # The binding finds libfa.so beside it; PyTorch's libraries are loaded before it (by importing torch).
    tmp = TORCH_LIB + ".tmp"
    _run(["g++", "-shared", "-o", tmp, torch_obj, "-L", os.path.join(_torch_dir(), "lib"), "-ltorch_python", "-ltorch",
          "-ltorch_cpu", "-ltorch_cuda", "-lc10", "-lc10_cuda", "-L", LIBDIR, "-l:libfa.so", "-Wl,-rpath,$ORIGIN"], "link of the binding")
    os.replace(tmp, TORCH_LIB)
    return LIB


if __name__ == "__main__":
    build(verbose="-v" in sys.argv, ptxas_info="--ptxas" in sys.argv)
    print(LIB)
