"""The attention's launch plan and layouts (csrc/decode_plan.hpp), checked on the host
by tests/sanitize/plan_driver.cpp."""
from __future__ import annotations

import os

import pytest

from test_sanitize_cpu import CLANGXX, HERE, _run


@pytest.fixture(scope="module")
def driver(tmp_path_factory):
    if not os.path.exists(CLANGXX):
        pytest.skip("clang++ is not available")
    exe = str(tmp_path_factory.mktemp("plan") / "plan_driver")
    _run([CLANGXX, "-O1", "-g", "-std=c++17", "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include",
          "-fsanitize=undefined", "-fno-sanitize-recover=all", os.path.join(HERE, "plan_driver.cpp"), "-o", exe])
    return exe


def test_plans_and_layouts(driver):
    assert "decode plan driver: ok" in _run([driver]).stdout
