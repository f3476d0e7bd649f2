"""Builds libnvfp4.so (the sm_100a CUDA kernels and their C ABI) in-tree, and
_fastcall, the compiled host path of the decode and gated calls, where torch and a
C++ compiler are there for it (without it those calls take the Python path).

    python -m w4a4_gemm_nvfp4_b200.build

nvcc cross-compiles for sm_100a without a GPU.  The CUDA runtime is linked
statically; the driver API (tensor-map encoding) is reached through
cudaGetDriverEntryPointByVersion, so the library does not link libcuda.
"""
from __future__ import annotations

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
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libnvfp4.so")
FAST = os.path.join(PKG, "_fastcall" + sysconfig.get_config_var("EXT_SUFFIX"))

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
COMMON = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC,-fvisibility=hidden", "-I", INCLUDE, "-I", CSRC]
# Per-file extra flags: the block step's arithmetic (quantizer kernels, and
# the GEMM epilogue that writes an NVFP4 output) must not be contracted into
# FMAs behind the explicit intrinsics' back.
EXTRA = {"quantize.cu": ["-fmad=false"], "gemm.cu": ["-fmad=false"]}
SOURCES = ["api.cu", "quantize.cu", "gemm.cu", "gemv.cu", "gated.cu"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _stale(target: str, deps: list[str]) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def build(verbose: bool = False, force: bool = False, ptxas_info: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    headers = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cuh", ".h"))]
    headers += [os.path.join(INCLUDE, f) for f in os.listdir(INCLUDE) if f.endswith(".h")]
    objs = []
    for src in SOURCES:
        path = os.path.join(CSRC, src)
        obj = os.path.join(BUILD, src.replace(".cu", ".o"))
        objs.append(obj)
        if force or _stale(obj, [path, *headers, __file__]):
            cmd = [nvcc(), *ARCH, *COMMON, *EXTRA.get(src, []), "-c", path, "-o", obj]
            if ptxas_info:
                cmd.insert(1, "-Xptxas=-v")
            if verbose:
                print(" ".join(cmd), flush=True)
            subprocess.run(cmd, check=True)
    if force or _stale(LIB, objs):
        tmp = LIB + f".tmp{os.getpid()}"
        cmd = [nvcc(), *ARCH, "-shared", "-o", tmp, *objs, "-cudart", "static"]
        if verbose:
            print(" ".join(cmd), flush=True)
        subprocess.run(cmd, check=True)
        os.replace(tmp, LIB)
    build_fastcall(verbose, force)
    return LIB


def torch_version() -> str:
    import torch

    return str(torch.__version__)


def build_fastcall(verbose: bool = False, force: bool = False) -> None:
    """The host-only extension module: the C++ compiler against this interpreter's
    and torch's headers, linked with libnvfp4.so beside it.  It is optional:
    without one of these a message says why, and no module is left behind.  It is
    built again for another Python or torch, whose classes it is compiled for."""
    untagged = os.path.join(PKG, "_fastcall.so")  # an earlier build's, which any Python would import
    if os.path.exists(untagged):
        os.remove(untagged)
    try:
        _build_fastcall(verbose, force)
    except (OSError, ImportError, subprocess.CalledProcessError) as e:
        if os.path.exists(FAST):
            os.remove(FAST)
        print(f"_fastcall (optional) is left out: {e}", file=sys.stderr)


def _build_fastcall(verbose: bool, force: bool) -> None:
    spec = importlib.util.find_spec("torch")
    if spec is None or not spec.origin:
        raise ImportError("torch is not installed")
    src, stamp = os.path.join(CSRC, "fastcall.cpp"), os.path.join(BUILD, "fastcall.stamp")
    built_for = torch_version()
    wanted = f"torch {built_for}, python {sys.version}"
    if not force and not _stale(FAST, [src, os.path.join(INCLUDE, "nvfp4.h"), __file__]) and os.path.exists(stamp):
        with open(stamp) as f:
            if f.read() == wanted:
                return
    cxx, include = os.environ.get("CXX", "g++"), sysconfig.get_paths()["include"]
    if not shutil.which(cxx):
        raise FileNotFoundError(f"no C++ compiler {cxx}")
    if not os.path.exists(os.path.join(include, "Python.h")):
        raise FileNotFoundError(f"no Python.h in {include}")
    torch_dir = os.path.dirname(spec.origin)
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))
    tmp = FAST + f".tmp{os.getpid()}"
    cmd = [cxx, "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden", "-Wall",
           f'-DBUILT_FOR="{built_for}"', "-I", INCLUDE, "-isystem", os.path.join(torch_dir, "include"),
           "-isystem", os.path.join(torch_dir, "include", "torch", "csrc", "api", "include"),
           "-isystem", os.path.join(cuda, "include"), "-I", include, src, "-o", tmp,
           "-L", PKG, "-lnvfp4", "-L", os.path.join(torch_dir, "lib"), "-ltorch_python", "-ltorch", "-ltorch_cpu",
           "-lc10", "-lc10_cuda", "-Wl,-rpath,$ORIGIN"]
    if verbose:
        print(" ".join(cmd), flush=True)
    try:
        subprocess.run(cmd, check=True)
        os.replace(tmp, FAST)
    finally:
        if os.path.exists(tmp):
            os.remove(tmp)
    os.makedirs(BUILD, exist_ok=True)
    with open(stamp, "w") as f:
        f.write(wanted)


if __name__ == "__main__":
    build(verbose=True, force="--force" in sys.argv, ptxas_info="-v" in sys.argv)
