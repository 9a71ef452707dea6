"""Ahead-of-time build of the HIP library ``libfp8lin.so`` for gfx950.

Every HIP source under ``csrc/`` is compiled with hipcc (in parallel), then
linked into one shared library next to this file; ``marshal.cpp`` becomes the
Python module ``_marshal.so`` beside it (host code only, against torch's headers).  No fast-math and no
denormal flushing: the quantizers rely on IEEE fp32 division with fp32
subnormals.  Packed fp32 VALU instructions are turned off for all device code.
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import subprocess
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(os.path.dirname(HERE), "include")
LIB = os.path.join(HERE, "libfp8lin.so")
MARSHAL = os.path.join(HERE, "_marshal.so")
BUILD_DIR = os.path.join(HERE, "_build")
SOURCES = ["api.hip", "quant.hip", "prune24.hip", "gemm_dense.hip", "gemm_sparse.hip", "workspace.hip",
           "fixed_scratch.hip", "api_layer.hip", "norm.hip", "kv_append.hip", "paged_decode.hip",
           "prompt_attention.hip"]

HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
ARCH = "gfx950"
CFLAGS = [
    f"--offload-arch={ARCH}", "-O3", "-std=c++17", "-fPIC", "-Wall", "-Wno-unused-result",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-fno-gpu-flush-denormals-to-zero", "-fhip-fp32-correctly-rounded-divide-sqrt",
    "-I", INCLUDE,
]


def _compile(src: str) -> str:
    obj = os.path.join(BUILD_DIR, os.path.splitext(src)[0] + ".o")
    cmd = [HIPCC, *CFLAGS, "-c", os.path.join(CSRC, src), "-o", obj]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"hipcc failed on {src}:\n{res.stderr}")
    return obj


def _compile_marshal() -> str:
    import torch
    from torch.utils.cpp_extension import include_paths

    obj = os.path.join(BUILD_DIR, "marshal.o")
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-Wall", "-D__HIP_PLATFORM_AMD__", "-DUSE_ROCM",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", "-I", INCLUDE,
           "-isystem", sysconfig.get_paths()["include"], "-isystem", "/opt/rocm/include"]
    for path in include_paths():
        cmd += ["-isystem", path]
    res = subprocess.run([*cmd, "-c", os.path.join(CSRC, "marshal.cpp"), "-o", obj], capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"g++ failed on marshal.cpp:\n{res.stderr}")
    return obj


def _link_marshal(obj: str) -> None:
    import torch

    tmp = MARSHAL + ".tmp%d" % os.getpid()
    cmd = ["g++", "-shared", obj, "-o", tmp, "-L", HERE, "-l:libfp8lin.so",
           "-L", os.path.join(os.path.dirname(torch.__file__), "lib"), "-lc10", "-ltorch_cpu", "-ltorch_hip", "-ltorch_python",
           "-Wl,-rpath,$ORIGIN"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"link of _marshal.so failed:\n{res.stderr}")
    os.replace(tmp, MARSHAL)


def build(verbose: bool = False) -> str:
    """Compile and link; returns the path of the shared library."""
    os.makedirs(BUILD_DIR, exist_ok=True)
    with cf.ThreadPoolExecutor(max_workers=min(len(SOURCES) + 1, os.cpu_count() or 4)) as ex:
        marshal = ex.submit(_compile_marshal)
        objs = list(ex.map(_compile, SOURCES))
    tmp = LIB + ".tmp%d" % os.getpid()
    cmd = [HIPCC, f"--offload-arch={ARCH}", "-shared", "-fPIC", *objs, "-o", tmp]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"link failed:\n{res.stderr}")
    os.replace(tmp, LIB)
    _link_marshal(marshal.result())  # last: the library alone serves the FP8 linears
    if verbose:
        print("built", LIB, "and", MARSHAL)
    return LIB


if __name__ == "__main__":
    build(verbose=True)
