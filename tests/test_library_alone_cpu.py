"""The library without the extension module of the decoder-layer calls: the FP8
linears' calls load and answer, and the decoder-layer calls say what is missing."""
from __future__ import annotations

import os
import shutil
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = """
import torch
import sparse_gemm_linears_amd as sgl
lib = sgl.load_library()
assert lib.fp8_quant_act(None, 4, 100, None, None, None) == sgl.FP8L_ERR_SHAPE
assert lib.fp8_quant_act(None, 4, 128, None, None, None) == sgl.FP8L_ERR_NULL
x = torch.zeros(2, 128, dtype=torch.bfloat16)
try:
    sgl.fp8_quant_act(x)
except ValueError as e:
    assert "device tensor" in str(e)
for _ in range(2):
    try:
        sgl.fp8_add_rmsnorm(x, x[0])
    except RuntimeError as e:
        assert "_marshal.so is missing" in str(e), e
    else:
        raise SystemExit("no error")
print("library alone: ok")
"""


def test_linears_need_the_library_alone(tmp_path):
    package = tmp_path / "sparse_gemm_linears_amd"
    package.mkdir()
    source = os.path.join(ROOT, "sparse_gemm_linears_amd")
    for name in ("__init__.py", "_binding.py", "libfp8lin.so"):
        shutil.copy(os.path.join(source, name), package / name)
    res = subprocess.run([sys.executable, "-c", PROGRAM], capture_output=True, text=True, cwd=tmp_path, timeout=300,
                         env=dict(os.environ, PYTHONPATH=str(tmp_path)))
    assert res.returncode == 0 and "library alone: ok" in res.stdout, res.stdout + res.stderr
