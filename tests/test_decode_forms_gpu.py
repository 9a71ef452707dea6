"""The forms of the attention that a launch plan chooses between, each against the
64-bit reference (attend_case of test_layer_gpu.py, with its tolerances)."""
from __future__ import annotations

import pytest
import torch

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


@pytest.mark.parametrize("lens,max_len", [([7], 32), ([40, 3], 4096), ([900] * 40, 4096)])
def test_infinite_values_stay_in_their_place(gpu_lib, lens, max_len):
    """An infinite value of a token that counts: an infinity or NaN in its own place of the row's heads, and nothing
    else moves."""
    g = torch.Generator(device="cuda").manual_seed(5)
    B, hq, hkv, d, page = len(lens), 8, 2, 128, 16
    per = max_len // page
    k, v = (torch.randn(B * per, hkv, page, d, generator=g, device="cuda").bfloat16() for _ in range(2))
    q = torch.randn(B, hq, d, generator=g, device="cuda").bfloat16()
    pages = torch.arange(B * per, dtype=torch.int32, device="cuda").view(B, per)
    seq = torch.tensor(lens, dtype=torch.int32, device="cuda")
    want = gpu_lib.paged_decode_attention(q, k, v, pages, seq)
    v[0, 1, 2, 77] = float("inf")  # token 2 of the first sequence, its second key head
    got = gpu_lib.paged_decode_attention(q, k, v, pages, seq)
    assert not torch.isfinite(got[0, 4:, 77]).any()
    got[0, 4:, 77] = want[0, 4:, 77]
    assert torch.equal(got, want)


@pytest.mark.parametrize("lens,max_len", [([9], 32), ([700, 3, 0], 4096), ([900] * 40, 4096)])
def test_values_of_any_size(gpu_lib, lens, max_len):
    """Values times a power of two give outputs times it, bit for bit, within the stated range and down to where the
    weights' second parts stay normal."""
    g = torch.Generator(device="cuda").manual_seed(6)
    B, hq, hkv, d, page = len(lens), 6, 2, 64, 16
    per = max_len // page
    k, v = (torch.randn(B * per, hkv, page, d, generator=g, device="cuda").bfloat16() for _ in range(2))
    v = torch.where(v.abs() < 2.0 ** -6, torch.full_like(v, 0.25), v)
    q = torch.randn(B, hq, d, generator=g, device="cuda").bfloat16()
    pages = torch.arange(B * per, dtype=torch.int32, device="cuda").view(B, per)
    seq = torch.tensor(lens, dtype=torch.int32, device="cuda")
    want, lse = gpu_lib.paged_decode_attention(q, k, v, pages, seq, return_lse=True)
    for power in (2.0 ** 105, 2.0 ** -40):  # below 8 x 2^105 x 900 tokens < 2^120
        got, again = gpu_lib.paged_decode_attention(q, k, v * power, pages, seq, return_lse=True)
        assert torch.isfinite(got).all() and torch.equal(got, want * power) and torch.equal(again, lse)
