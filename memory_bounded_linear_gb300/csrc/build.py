"""Build ``liblce.so`` (the C-ABI library) for sm_103a with nvcc, and ``_native.so`` (its binding to
torch tensors for the operators called once per layer and token) with the host compiler, in-tree.
liblce.so needs nothing but nvcc: it is linked first, and without torch the binding is left out.

Each translation unit is compiled in parallel to an object file under ``_build/`` at the
repository root, then linked (CUDA runtime linked statically) into
``memory_bounded_linear_gb300/liblce.so``.  Usage: ``python -m memory_bounded_linear_gb300.csrc.build``,
or without torch, which the package imports, ``python memory_bounded_linear_gb300/csrc/build.py``.
"""

from __future__ import annotations

import concurrent.futures as cf
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

CSRC = os.path.dirname(os.path.abspath(__file__))
PKG = os.path.dirname(CSRC)
ROOT = os.path.dirname(PKG)
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "liblce.so")
NATIVE = os.path.join(PKG, "_native.so")

SOURCES = ["lce_api.cu", "lce_tc.cu", "lce_simt.cu", "lce_reduce.cu", "lce_static_scratch.cu",
           "lce_ffn_api.cu", "lce_ffn_few.cu", "lce_ffn_simt.cu", "lce_ffn_tc.cu",
           "lce_gradnorm.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall",
         f"-I{INCLUDE}", f"-I{CSRC}"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found (set NVCC or put CUDA's bin directory on PATH)")


def _compile(src: str, ptxas_verbose: bool) -> tuple[str, str]:
    obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
    cmd = [nvcc(), *ARCH, *FLAGS, "-c", os.path.join(CSRC, src), "-o", obj]
    if ptxas_verbose:
        cmd += ["-Xptxas", "-v"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed for {src}:\n{' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    return obj, r.stdout + r.stderr


def _compile_binding() -> str | None:
    """Object file of the binding, None without torch; torch's headers and its C++ ABI come from the
    installed torch."""
    if importlib.util.find_spec("torch") is None:
        return None
    import torch
    from torch.utils import cpp_extension

    obj = os.path.join(BUILD, "py_binding.o")
    include = [INCLUDE, *cpp_extension.include_paths("cuda"), sysconfig.get_paths()["include"]]
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-Wall",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}",
           *[f"-isystem{i}" for i in include],
           "-c", os.path.join(CSRC, "py_binding.cpp"), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed for py_binding.cpp:\n{' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    return obj


def _link_binding(obj: str) -> None:
    from torch.utils import cpp_extension

    tmp = NATIVE + ".tmp"
    cmd = [os.environ.get("CXX", "g++"), "-shared", "-o", tmp, obj, LIB, "-Wl,-rpath,$ORIGIN",
           *[f"-L{p}" for p in cpp_extension.library_paths("cuda")],
           "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10", "-lc10_cuda"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link of the binding failed:\n{' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, NATIVE)


def build(verbose: bool = False, ptxas_verbose: bool = False) -> str:
    """Compile every source for sm_103a, link liblce.so and its binding; returns the library path."""
    os.makedirs(BUILD, exist_ok=True)
    with cf.ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        binding = ex.submit(_compile_binding)
        results = list(ex.map(lambda s: _compile(s, ptxas_verbose), SOURCES))
    objs = [o for o, _ in results]
    if verbose:
        for (_, log), src in zip(results, SOURCES):
            if log.strip():
                print(f"--- {src}\n{log}")
    tmp = LIB + ".tmp"
    cmd = [nvcc(), *ARCH, "-shared", "-cudart", "static", "-Xlinker", "-soname=liblce.so", "-o", tmp,
           *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    obj = binding.result()
    if obj is None:
        print("torch is not installed: _native.so, the binding to its tensors, is not built", file=sys.stderr)
    else:
        _link_binding(obj)
    return LIB


if __name__ == "__main__":
    print(build(verbose=True, ptxas_verbose="-v" in sys.argv))
