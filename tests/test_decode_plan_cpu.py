"""The attention's launch plan and layouts (csrc/decode_plan.hpp), checked on the host
by tests/sanitize/plan_driver.cpp."""
from __future__ import annotations

import os

import pytest

from decode_forms import BATCHES
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


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("batch", BATCHES, ids=lambda b: b.name)
def test_batches_reach_their_forms(driver, batch, fp8):
    """Each batch of test_decode_forms_gpu.py takes the form it is there for, whatever the plan's thresholds are."""
    args = (batch.B, batch.Hq, batch.Hkv, batch.D, int(fp8), batch.max_len, batch.window)
    waves, splits, by_row = (int(x) for x in _run([driver, *map(str, args)]).stdout.split())
    if waves:
        assert batch.form == ("rows", waves, splits > 1)
    else:
        assert batch.form == ("shares", "listed by row" if by_row else "by share")
    assert len(batch.lens()) == batch.B and max(batch.lens()) <= batch.max_len
    assert not batch.window or batch.window >= 1000 or max(batch.lens()) > batch.window
