"""Outputs that the binding allocates are laid out as torch.empty lays them out, whatever
the strides of the input's dimensions of one element (which a contiguous tensor may
have) and with dimensions of none."""
from __future__ import annotations

import pytest
import torch

from sparse_gemm_linears_amd import _binding


@pytest.mark.parametrize("shape", [(1, 128), (1, 1, 256), (3, 128), (128,), (0, 128), (4, 0), (2, 0, 8), (1, 0)])
def test_allocated_outputs_are_laid_out_plainly(shape):
    want = torch.empty(shape).stride()
    odd = [s * 999 if n == 1 else s for n, s in zip(shape, want)]
    same = torch.empty_strided(shape, odd, dtype=torch.bfloat16)
    other = torch.empty(7, 5, dtype=torch.bfloat16)
    for like in (same, other):
        assert like.is_contiguous()
        out = _binding._out(None, "q", shape, torch.uint8, like)
        assert out.dtype == torch.uint8 and out.shape == shape and out.stride() == want
    row = torch.empty(6, 999, dtype=torch.bfloat16)[2:3, :128]  # one row of a wider matrix
    assert row.is_contiguous()
    q = _binding._out(None, "q", (1, 128), torch.uint8, row)
    assert q.view(torch.int32).shape == (1, 32)
