"""Build libgdn.so (the HIP library behind include/gdn.h) for gfx950 in-tree.

    python -m chunked_gated_delta_05_amd.build [-v]

hipcc compiles the kernels and the host API into one shared library next to
this file, and g++ the torch marshalling of the recurrent-state operators
(_native.so). Packed FP32 instructions are disabled for all device code.
"""
from __future__ import annotations

import os
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libgdn.so")
NATIVE = os.path.join(HERE, "_native.so")
SOURCES = [os.path.join(CSRC, "gdn_kernels.hip"), os.path.join(CSRC, "gdn_host.cpp"),
           os.path.join(CSRC, "gdn_noalloc.hip"), os.path.join(CSRC, "gdn_bwd.hip")]
# the recurrent-state operators of include/gdn_recurrent.h
RECURRENT_HIP = ["gdn_linattn", "gdn_step", "gdn_pages"]
RECURRENT_HOST = "gdn_recurrent_host"
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")


BUILD = os.path.join(HERE, "_build")


def _run(cmd, verbose):
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.run(cmd, check=True)


def build(verbose: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    inc = ["-I", os.path.join(ROOT, "include"), "-I", CSRC]
    warn = ["-Wall", "-Wno-unused-function", "-Wno-unused-variable"]
    kobj = os.path.join(BUILD, "gdn_kernels.o")
    hobj = os.path.join(BUILD, "gdn_host.o")
    nobj = os.path.join(BUILD, "gdn_noalloc.o")
    bobj = os.path.join(BUILD, "gdn_bwd.o")
    _run([HIPCC, "--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC",
          "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
          # MFMA accumulators in ordinary VGPRs: the state update scales them
          # with VALU ops every chunk, which AGPR accumulators turn into copies
          "-mllvm", "-amdgpu-mfma-vgpr-form=1",
          *warn, *inc, "-c", SOURCES[0], "-o", kobj], verbose)
    _run([HIPCC, "-O2", "-std=c++17", "-fPIC", "-D__HIP_PLATFORM_AMD__", *warn, *inc, "-I", "/opt/rocm/include",
          "-x", "c++", "-c", SOURCES[1], "-o", hobj], verbose)
    _run([HIPCC, "--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC",
          "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
          *warn, *inc, "-c", SOURCES[2], "-o", nobj], verbose)
    _run([HIPCC, "--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC",
          "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
          *warn, *inc, "-c", SOURCES[3], "-o", bobj], verbose)
    robjs = []
    for name in RECURRENT_HIP:
        robjs.append(os.path.join(BUILD, name + ".o"))
        # MFMA accumulators in ordinary VGPRs, as above: the state is scaled
        # and split by VALU ops every chunk
        _run([HIPCC, "--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC",
              "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops", "-mllvm", "-amdgpu-mfma-vgpr-form=1",
              *warn, *inc, "-c", os.path.join(CSRC, name + ".hip"), "-o", robjs[-1]], verbose)
    robjs.append(os.path.join(BUILD, RECURRENT_HOST + ".o"))
    _run([HIPCC, "-O2", "-std=c++17", "-fPIC", "-D__HIP_PLATFORM_AMD__", *warn, *inc, "-I", "/opt/rocm/include",
          "-x", "c++", "-c", os.path.join(CSRC, RECURRENT_HOST + ".cpp"), "-o", robjs[-1]], verbose)
    _run([HIPCC, "--offload-arch=gfx950", "-shared", "-fPIC", kobj, hobj, nobj, bobj, *robjs, "-o", LIB + ".tmp"],
         verbose)
    os.replace(LIB + ".tmp", LIB)
    _build_native(inc, verbose)
    return LIB


def _build_native(inc, verbose):
    """_native.so: torch marshalling of the recurrent-state operators (host
    code; CPython's C API and torch's C++ headers)."""
    import torch
    from torch.utils.cpp_extension import include_paths, library_paths

    tinc = [x for p in include_paths() for x in ("-isystem", p)]
    tlib = [x for p in library_paths() for x in ("-L" + p, "-Wl,-rpath," + p)]
    _run(["g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-fvisibility=hidden", "-D__HIP_PLATFORM_AMD__", "-DUSE_ROCM",
          f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", *inc, *tinc,
          "-isystem", sysconfig.get_path("include"), "-isystem", "/opt/rocm/include",
          os.path.join(CSRC, "gdn_torch.cpp"), "-o", NATIVE + ".tmp",
          "-L" + HERE, "-l:libgdn.so", "-Wl,-rpath,$ORIGIN", *tlib, "-lc10", "-lc10_hip", "-ltorch_cpu",
          "-ltorch_python"], verbose)
    os.replace(NATIVE + ".tmp", NATIVE)


if __name__ == "__main__":
    build(verbose="-v" in sys.argv)
