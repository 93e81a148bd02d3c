"""Builds libhc.so in-tree from csrc/ with hipcc for gfx950.

Flags: -O3, -ffp-contract=off (no fused multiply-add contraction: every hop is
one IEEE add), no fast-math, no flush-to-zero, packed-fp32 instructions
disabled on the device (-Xclang -target-feature -Xclang -packed-fp32-ops).
Objects go to _build/ at the repository root; the library lands next to this
file so that it travels with the tree.  The two measurement programs of
measure/ at the repository root are built there: dma_contention (linked
against libhc and rocBLAS from the system ROCm) and hbm_ceiling.

Beside the library lands _native.so, the module that marshals torch tensors to
it for calls where Python's share would be the larger.  It needs torch, its and
Python's headers and a host compiler, which the library and the programs do
not: they are built whatever becomes of it, and where one of these is missing
it is left out with a message (the binding's calls that go through it then
raise ImportError).
"""
from __future__ import annotations

import concurrent.futures as cf
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
LIB = os.path.join(PKG, "libhc.so")
NATIVE = os.path.join(PKG, "_native.so")
MEASURE = os.path.join(ROOT, "measure")
DMA_TOOL = os.path.join(MEASURE, "dma_contention")
CEILING_TOOL = os.path.join(MEASURE, "hbm_ceiling")
ARCH = os.environ.get("HC_OFFLOAD_ARCH", "gfx950")
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
CXX = os.environ.get("CXX", "g++")

SOURCES = ["hc_api.cpp", "schedule.cpp", "ring_kernels.hip", "codec_kernels.hip", "car_chain.hip",
           "entropy_kernels.hip", "step_api.cpp", "grad_kernels.hip", "embed_kernels.hip", "expert_kernels.hip"]

COMMON = ["-O3", "-std=c++17", "-fPIC", "-ffp-contract=off", "-fno-fast-math",
          "-Wall", "-Wno-unused-function", "-I", INCLUDE, "-I", CSRC]
DEVICE = [f"--offload-arch={ARCH}", "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
          "-fno-gpu-rdc"]


def _compile(src: str) -> str:
    obj = os.path.join(BUILD, os.path.basename(src) + ".o")
    cmd = [HIPCC, *COMMON, *DEVICE, "-x", "hip", "-c", os.path.join(CSRC, src), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"hipcc failed for {src}:\n{' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    return obj


def _native_lacks() -> str | None:
    """What _native.so needs that is not here, or None."""
    try:
        import torch
    except ImportError:
        return "torch"
    for path in (os.path.join(os.path.dirname(torch.__file__), "include", "torch", "csrc", "autograd",
                              "python_variable.h"),
                 os.path.join(sysconfig.get_paths()["include"], "Python.h")):
        if not os.path.exists(path):
            return path
    return None if shutil.which(CXX) else f"the compiler {CXX}"


def _compile_native() -> str:
    """native_binding.cpp, host code against torch's and Python's headers."""
    import torch

    inc = os.path.join(os.path.dirname(torch.__file__), "include")
    obj = os.path.join(BUILD, "native_binding.cpp.o")
    cmd = [CXX, "-O2", "-std=c++17", "-fPIC", "-Wall", "-Wno-unused-function", "-D__HIP_PLATFORM_AMD__", "-DUSE_ROCM",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", "-I", INCLUDE, "-isystem", inc,
           "-isystem", os.path.join(inc, "torch", "csrc", "api", "include"), "-isystem", "/opt/rocm/include",
           "-isystem", sysconfig.get_paths()["include"], "-c", os.path.join(CSRC, "native_binding.cpp"), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"compiler failed for native_binding.cpp:\n{' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    return obj


def _link_native(obj: str):
    """_native.so finds libhc.so beside it; torch's libraries are in the
    process that imports it."""
    import torch

    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    tmp = NATIVE + ".tmp"
    cmd = [CXX, "-shared", "-o", tmp, obj, "-L", PKG, "-lhc", "-Wl,-rpath,$ORIGIN", "-L", lib, "-ltorch_python",
           "-ltorch_cpu", "-lc10", "-lc10_hip"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, NATIVE)


def _build_tools():
    """The measurement programs."""
    tmp = DMA_TOOL + ".tmp"
    cmd = [HIPCC, *COMMON, *DEVICE, "-x", "hip", os.path.join(MEASURE, "dma_contention.hip"), "-o", tmp,
           "-L", PKG, "-lhc", "-Wl,-rpath,$ORIGIN/../collective_communication_amd", "-L/opt/rocm/lib", "-lrocblas", "-Wl,-rpath,/opt/rocm/lib"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"dma_contention build failed:\n{' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, DMA_TOOL)
    tmp = CEILING_TOOL + ".tmp"
    cmd = [HIPCC, *COMMON, *DEVICE, "-x", "hip", os.path.join(MEASURE, "hbm_ceiling.hip"), "-o", tmp]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"hbm_ceiling build failed:\n{' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, CEILING_TOOL)


def build(verbose: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    lacks = _native_lacks()
    jobs = min(len(SOURCES) + 1, max(1, min(8, os.cpu_count() or 1)))
    with cf.ThreadPoolExecutor(jobs) as ex:
        native = None if lacks else ex.submit(_compile_native)
        objs = list(ex.map(_compile, SOURCES))
    tmp = LIB + ".tmp"
    cmd = [HIPCC, f"--offload-arch={ARCH}", "-shared", "-fPIC", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    done = False
    try:
        if native:
            _link_native(native.result())
            done = True
        else:
            print(f"_native.so is not built: {lacks} is missing", file=sys.stderr)
    finally:
        if not done and os.path.exists(NATIVE):
            os.remove(NATIVE)     # of the library that was here before
        _build_tools()
    if verbose:
        print("built " + ", ".join(p for p in (LIB, None if lacks else NATIVE, DMA_TOOL, CEILING_TOOL) if p))
    return LIB


if __name__ == "__main__":
    build(verbose=True)
    sys.exit(0)
