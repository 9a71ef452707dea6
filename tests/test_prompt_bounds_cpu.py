"""What the launch plan of the attention of several tokens promises of its divisions: how many workgroups, and how many
bytes of partials (tests/sanitize/prompt_bound_driver.cpp, built with the sanitizers)."""
from __future__ import annotations

import os

import pytest

from test_sanitize_cpu import CLANGXX, HERE, _run


def test_divisions_stay_within_their_bounds(tmp_path):
    if not os.path.exists(CLANGXX):
        pytest.skip("clang++ is not available")
    exe = str(tmp_path / "prompt_bound_driver")
    _run([CLANGXX, "-O1", "-g", "-std=c++17", "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include",
          "-fsanitize=address,undefined", "-fno-sanitize-recover=all", os.path.join(HERE, "prompt_bound_driver.cpp"),
          "-o", exe])
    assert "prompt bounds: ok" in _run([exe], env=dict(os.environ, ASAN_OPTIONS="detect_leaks=0")).stdout
