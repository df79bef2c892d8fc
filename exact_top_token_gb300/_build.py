"""Compile the CUDA library (sm_103a) in-tree with nvcc: one object per
translation unit, compiled in parallel, linked into ``_build/libhytopk.so``;
and, where torch is installed, the operators' Python module against it with the
host compiler (``csrc/binding.cpp``)."""
from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(BUILD, "libhytopk.so")
BINDING_SRC = os.path.join(CSRC, "binding.cpp")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-O2",
              "-Xcompiler", "-fvisibility=hidden",
              "--expt-relaxed-constexpr", "-I", INCLUDE, "-I", CSRC]


def nvcc() -> str:
    home = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    cand = os.path.join(home, "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _inputs():
    return sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(
        os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(INCLUDE, "*.h")) + [__file__]


def _older(out, inputs) -> bool:
    return not os.path.exists(out) or any(
        os.path.getmtime(f) > os.path.getmtime(out) for f in inputs)


def stale() -> bool:
    return _older(LIB, _inputs())


def binding() -> str | None:
    """Path of the operators' Python module, built for this Python and this torch; None
    without torch (the library does not need it)."""
    try:
        import torch
    except ImportError:
        return None
    return os.path.join(BUILD, f"_operators-{torch.__version__}-{sys.implementation.cache_tag}.so")


def _build_binding(out):
    """Compile csrc/binding.cpp; it uses the torch libraries of the process."""
    import sysconfig

    import torch

    top = os.path.dirname(os.path.abspath(torch.__file__))
    cuda = os.path.dirname(os.path.dirname(nvcc())) or "/usr/local/cuda"
    include = [INCLUDE, os.path.join(top, "include"),
               os.path.join(top, "include", "torch", "csrc", "api", "include"),
               sysconfig.get_path("include"), os.path.join(cuda, "include")]
    tmp = out + f".tmp{os.getpid()}"
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared",
           "-fvisibility=hidden", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}",
           *(f"-I{i}" for i in include), BINDING_SRC, f"-L{os.path.join(top, 'lib')}", "-lc10",
           "-lc10_cuda", "-ltorch_cpu", "-ltorch_python", "-o", tmp]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{cmd[0]} failed on {os.path.basename(BINDING_SRC)}:\n{r.stderr}")
    os.replace(tmp, out)


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    """Build the library and (with torch) the operators' module if missing or out of date;
    returns the library's path. A module that does not build raises when the library is
    there."""
    os.makedirs(BUILD, exist_ok=True)
    module = binding()
    if module and not force and not _older(
            module, [BINDING_SRC, os.path.join(INCLUDE, "hytopk.h"), __file__]):
        module = None
    with cf.ThreadPoolExecutor(max_workers=1) as ex:
        other = ex.submit(_build_binding, module) if module else None
        if force or stale():
            _build_library(verbose, extra_flags)
        if other is not None:
            other.result()
    return LIB


def _build_library(verbose, extra_flags):
    srcs = sources()
    objs = [os.path.join(BUILD, os.path.basename(s)[:-3] + ".o") for s in srcs]

    def compile_one(src_obj):
        src, obj = src_obj
        cmd = [nvcc(), *ARCH, *NVCC_FLAGS, *extra_flags, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {os.path.basename(src)}:\n{r.stderr}")
        return r.stderr

    with cf.ThreadPoolExecutor(max_workers=min(16, len(srcs))) as ex:
        logs = list(ex.map(compile_one, zip(srcs, objs)))
    if verbose:
        for s, log in zip(srcs, logs):
            if log.strip():
                print(f"[{os.path.basename(s)}]\n{log}")
    tmp = LIB + f".tmp{os.getpid()}"
    r = subprocess.run([nvcc(), *ARCH, "-shared", "-o", tmp, *objs], capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stderr}")
    os.replace(tmp, LIB)
