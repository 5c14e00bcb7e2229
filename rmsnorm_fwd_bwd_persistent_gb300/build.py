"""Builds the CUDA library ``librmsn_gb300.so`` in-tree for sm_103a with nvcc, and the
CPython module ``_binding.so`` (the tensor side of the attention entry points) with g++.

The translation units compile in parallel (one compiler per file) and are linked into one
shared library with the CUDA runtime linked statically, so the library depends only on
the driver.  No fast-math: IEEE division and square root, no flush-to-zero.  The module is
linked against the library and the torch it is built with.

Usage: ``python -m rmsnorm_fwd_bwd_persistent_gb300.build [--verbose-ptxas]``
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "librmsn_gb300.so")

BINDING = os.path.join(PKG, "_binding.so")
BINDING_SOURCE = "rmsn_binding.cpp"

SOURCES = ["rmsn_api.cu", "rmsn_fwd.cu", "rmsn_bwd.cu", "rmsn_bwd_small.cu",
           "rmsn_fused_quant.cu", "rmsn_qk.cu", "rmsn_kv4.cu", "rmsn_kv4_attn.cu",
           "rmsn_attn_api.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ARCH + [
    "-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC,-O2",
    "--prec-div=true", "--prec-sqrt=true", "--ftz=false", "--fmad=true",
    "-I", INCLUDE, "-I", CSRC,
]


def _nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build the library")


def _deps() -> list[str]:
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC)]
    files.append(os.path.join(INCLUDE, "rmsn.h"))
    files.append(os.path.abspath(__file__))
    return files


def up_to_date() -> bool:
    if not (os.path.exists(LIB) and os.path.exists(BINDING)):
        return False
    t = min(os.path.getmtime(LIB), os.path.getmtime(BINDING))
    return all(os.path.getmtime(f) <= t for f in _deps())


def _binding_flags() -> tuple[list[str], list[str]]:
    """Compile and link flags of the module: the headers and libraries of the installed torch."""
    import sysconfig

    import torch
    base = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(_nvcc())))
    lib = os.path.join(base, "lib")
    compile_ = ["-O2", "-std=c++17", "-fPIC", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
                "-I", INCLUDE, "-isystem", os.path.join(base, "include"),
                "-isystem", os.path.join(cuda, "include"),
                "-isystem", sysconfig.get_paths()["include"]]
    link = ["-L", lib, "-ltorch_python", "-ltorch", "-ltorch_cpu", "-ltorch_cuda", "-lc10", "-lc10_cuda",
            "-L", PKG, "-l:" + os.path.basename(LIB), "-Wl,-rpath,$ORIGIN"]
    return compile_, link


def _run(cmd: list[str], what: str) -> str:
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{what} failed:\n{r.stdout}\n{r.stderr}")
    return r.stderr


def build(force: bool = False, verbose_ptxas: bool = False, jobs: int | None = None) -> str:
    if not force and up_to_date():
        return LIB
    nvcc = _nvcc()
    os.makedirs(BUILD, exist_ok=True)
    extra = ["-Xptxas", "-v"] if verbose_ptxas else []

    cxx = shutil.which("g++") or "g++"
    cxx_flags, cxx_link = _binding_flags()

    def compile_one(src: str) -> tuple[str, str]:
        obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
        path = os.path.join(CSRC, src)
        cmd = [cxx, *cxx_flags, "-c", path, "-o", obj] if src == BINDING_SOURCE else \
            [nvcc, *NVCC_FLAGS, *extra, "-c", path, "-o", obj]
        return obj, _run(cmd, f"compiling {src}")

    sources = SOURCES + [BINDING_SOURCE]
    with cf.ThreadPoolExecutor(max_workers=jobs or len(sources)) as ex:
        results = list(ex.map(compile_one, sources))
    if verbose_ptxas:
        for (_, log) in results:
            sys.stderr.write(log)
    objs = [o for o, _ in results]
    tmp = LIB + f".tmp{os.getpid()}"
    _run([nvcc, *ARCH, "-shared", "-cudart", "static", "-o", tmp, *objs[:-1]], "linking the library")
    os.replace(tmp, LIB)
    tmp = BINDING + f".tmp{os.getpid()}"
    _run([cxx, "-shared", "-o", tmp, objs[-1], *cxx_link], "linking the module")
    os.replace(tmp, BINDING)
    return LIB


if __name__ == "__main__":
    build(force=True, verbose_ptxas="--verbose-ptxas" in sys.argv)
    print(LIB)
