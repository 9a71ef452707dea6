"""Attention of several tokens whose scale and cap lie far apart (tolerances in prompt_ref.py)."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import layer_ref as ref
from prompt_ref import Check, heads
from test_layer_gpu import gen
from test_prompt_gpu import starts_of

pytestmark = pytest.mark.gpu

FAR = [(1e10, 1e-29), (-1e10, 1e-45), (2.0 ** 100, 1e-30), (2.0 ** 100, 5.0),  # caps that no score is below
       (1e-3, 1e38), (1e-6, 3e38), (1e-12, 1e30), (1e-30, 1e12), (1e-33, 1e8)]  # caps that no score comes near


@pytest.mark.parametrize("scale,softcap", FAR)
@pytest.mark.parametrize("D", [64, 128])
def test_scale_and_cap_far_apart(gpu_lib, D, scale, softcap):
    """Scores of a softmax's usual size where the scale is small (queries and keys share the rest), any where it is
    large; a head of zero queries has scores of exactly 0."""
    r = gen("far", D, abs(scale), softcap)
    n, Hq, Hkv = 140, 3, 1
    size = min(1.0, abs(scale)) ** -0.5 / D ** 0.25
    q = ref.bf16(size * r.standard_normal((n, Hq, D)))
    q[:, 1] = 0
    k = ref.bf16(size * r.standard_normal((n, Hkv, D)))
    v = ref.bf16(r.standard_normal((n, Hkv, D)))
    scale, softcap = (float(np.float32(x)) for x in (scale, softcap))
    o, lse = gpu_lib.prompt_attention(q.cuda(), k.cuda(), v.cuda(), starts_of([n]), scale=scale, softcap=softcap,
                                      return_lse=True)
    many = Check(scale, softcap)
    many.sequence(o, lse, ref.f64(q), heads(k), heads(v), 0, what="of a prompt")
    # the last tokens over a cache of one page
    cache = [torch.nn.functional.pad(x.transpose(0, 1), (0, 0, 0, 144 - n))[None].contiguous().cuda() for x in (k, v)]
    o, lse = gpu_lib.paged_chunk_attention(q[-5:].cuda(), *cache, torch.zeros(1, 1, dtype=torch.int32, device="cuda"),
                                           torch.tensor([n], dtype=torch.int32, device="cuda"), starts_of([5]),
                                           scale=scale, softcap=softcap, return_lse=True)
    few = Check(scale, softcap)
    few.sequence(o, lse, ref.f64(q[-5:]), heads(k), heads(v), n - 5, what="of a chunk")
