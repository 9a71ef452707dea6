"""Batches on either side of the sizes up to which lengths divide a batch, one sequence of it far longer than the rest
(tolerances in prompt_ref.py)."""
from __future__ import annotations

import pytest
import torch

import layer_ref as ref
from prompt_ref import Check
from test_chunk_gpu import shared_pages
from test_layer_gpu import gen
from test_prompt_gpu import starts_of

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("B,new,Hq,Hkv,D", [(62, 4, 32, 32, 64), (64, 4, 32, 32, 64), (228, 4, 32, 8, 128), (229, 4, 32, 8, 128),
                                            (256, 1, 4, 2, 128), (257, 1, 4, 2, 128), (257, 3, 2, 2, 256)])
def test_one_long_sequence(gpu_lib, B, new, Hq, Hkv, D, fp8):
    length, page = 9000, 16
    cache, row, (k, v) = shared_pages(D, Hkv, length, page, fp8, B)
    lens = [1 + (b * 37) % 300 for b in range(B)]
    long = B // 3
    lens[long] = length
    q = ref.bf16(1.5 * gen("one long", B, D).standard_normal((B * new, Hq, D)))
    call = gpu_lib.paged_chunk_attention_fp8 if fp8 else gpu_lib.paged_chunk_attention
    args = (q.cuda(), *cache, row.expand(B, -1).contiguous(), torch.tensor(lens, dtype=torch.int32, device="cuda"),
            starts_of([new] * B))
    o, lse = call(*args, return_lse=True)
    check = Check(D ** -0.5, 0.0)
    for b in (0, 1, long - 1, long, long + 1, B - 1):
        rows = slice(b * new, (b + 1) * new)
        check.sequence(o[rows], lse[rows], ref.f64(q[rows]), k[:, : lens[b]], v[:, : lens[b]], lens[b] - new,
                       what=f"of sequence {b}, {lens[b]} tokens")
    check.done()
    assert torch.equal(call(*args), o)
