"""The forms of the attention that a launch plan chooses between, each against the
64-bit reference (attend_case of test_layer_gpu.py, with its tolerances)."""
from __future__ import annotations

import pytest

from decode_forms import BATCHES
from test_layer_gpu import attend_case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("Hq,Hkv,D", [(1, 1, 64), (3, 1, 64), (35, 5, 64), (15, 1, 64), (5, 1, 128), (28, 4, 128),
                                      (33, 3, 128), (3, 3, 256), (9, 3, 256), (13, 1, 256), (16, 2, 128)])
def test_one_wave_rows(gpu_lib, Hq, Hkv, D, fp8):
    """Rows of one tile at most, which a workgroup of one wave takes, with odd numbers of query heads on a key head
    too: by a bound of 32 tokens, and by windows whose tokens lie in one tile."""
    attend_case(gpu_lib, [0, 1, 2, 15, 16, 17, 30, 31, 32], Hq, Hkv, D, 16, fp8, max_len=32)
    attend_case(gpu_lib, [0, 1, 16, 17, 33, 47, 100, 161], Hq, Hkv, D, 16, fp8, window=17)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("batch", BATCHES, ids=lambda b: b.name)
def test_forms(gpu_lib, batch, fp8):
    """Ragged batches with empty sequences through each form: even shares that list divided rows by row or by share,
    with and without a window, and short rows in workgroups of one, two and four waves."""
    attend_case(gpu_lib, batch.lens(), batch.Hq, batch.Hkv, batch.D, batch.page, fp8, window=batch.window,
                max_len=batch.max_len)
