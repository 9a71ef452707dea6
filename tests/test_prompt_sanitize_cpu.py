"""Address and undefined-behaviour sanitizer run of the prompt and chunk calls' host code
(tests/sanitize/prompt_driver.cpp): built with the sanitizers on the host side only and
driven without a GPU."""
from __future__ import annotations

import os
import subprocess

import pytest

from sparse_gemm_linears_amd.build import SOURCES
from test_sanitize_cpu import CLANGXX, CSRC, HERE, HIPCC, ROOT, _run


def test_prompt_host_code_under_sanitizers(tmp_path):
    if not (os.path.exists(HIPCC) and os.path.exists(CLANGXX)):
        pytest.skip("hipcc / clang++ are not available")
    procs = []
    for src in SOURCES:
        obj = str(tmp_path / (src[:-4] + ".o"))
        # sanitizers on the host side only; the device code as in the product build
        cmd = [HIPCC, "--offload-arch=gfx950", "-O1", "-g", "-std=c++17", "-fPIC",
               "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
               "-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
               "-Xarch_host", "-fno-sanitize-recover=all",
               "-I", os.path.join(ROOT, "include"), "-c", os.path.join(CSRC, src), "-o", obj]
        procs.append((obj, cmd, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.PIPE, text=True)))
    for _, cmd, p in procs:
        _, err = p.communicate(timeout=600)
        assert p.returncode == 0, f"{' '.join(cmd)}\n{err}"
    exe = str(tmp_path / "prompt_driver")
    _run([CLANGXX, "-O1", "-g", "-std=c++17", "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include",
          "-fsanitize=address,undefined", "-fno-sanitize-recover=all", os.path.join(HERE, "prompt_driver.cpp"),
          *[o for o, _, _ in procs], "-L/opt/rocm/lib", "-lamdhip64", "-Wl,-rpath,/opt/rocm/lib", "-o", exe])
    res = _run([exe], env=dict(os.environ, ASAN_OPTIONS="detect_leaks=0"))
    assert "prompt host sanitizer driver: ok" in res.stdout
