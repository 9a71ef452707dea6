"""Attention of several tokens with scores far beyond a softmax's usual range: one key takes all the weight.

Each query and key has one value that is not zero, so that a product q.k has 16 bits and is exact in fp32; the keys'
values differ by 2^-8 of themselves at least, so that the second largest score is 2^12 below the largest or more and its
weight is 0.  o is the value of the key with the largest score, within the weight's one bf16 (2^-8) and a product in fp32
before its own rounding.  The score takes six roundings to fp32 on its way to lse (log2 e and its product with the scale,
the product, and the same of ln 2): 2^-21 of it and 2^-18; under a cap 2^-19 more, as in prompt_ref.py.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

import layer_ref as ref
from test_layer_gpu import U, assert_rounded, gen, holds
from test_prompt_gpu import starts_of

pytestmark = pytest.mark.gpu


def one_value_each(tokens, keys, Hq, Hkv, D, seed):
    """Queries' values [tokens, Hq] of both signs, keys' [Hkv, keys], all distinct, and values [Hkv, keys, D]."""
    r = gen("large", tokens, keys, Hq, Hkv, D, seed)
    steps = np.concatenate([(1 + np.arange(128) / 128) * 2.0 ** j for j in range(4)])
    a = r.choice(steps, (tokens, Hq)) * r.choice([-1.0, 1.0], (tokens, Hq))
    b = np.stack([r.permutation(steps)[:keys] for _ in range(Hkv)])
    return a, b, r.standard_normal((Hkv, keys, D))


def hold_to_the_largest(o, lse, a, b, v, scale, softcap):
    """a of the last tokens of a sequence with keys b [Hkv, keys] and values v [Hkv, keys, D]."""
    tokens, hq = a.shape
    hkv, keys = b.shape
    want, score = np.zeros((tokens, hq, v.shape[-1])), np.zeros((tokens, hq))
    for t in range(tokens):
        for h in range(hq):
            kvh = h // (hq // hkv)
            s = scale * a[t, h] * b[kvh, : keys - tokens + t + 1]
            want[t, h], score[t, h] = v[kvh, s.argmax()], s.max()
    if softcap:
        score = softcap * np.tanh(score / softcap)
    assert_rounded(o, want, (2.0 ** -8 * (1 + 2.0 ** -8) + 2 * U) * np.abs(want), "o")
    holds(np.abs(ref.f64(lse) - score) <= (2.0 ** -21 + (2.0 ** -19 if softcap else 0)) * np.abs(score) + 2.0 ** -18,
          "lse")


SCALES = [1.1 * 2 ** 20, 1.3 * 2 ** 27, -1.234 * 2 ** 31, 1.7 * 2 ** 40, 1.3 * 2 ** 95]


@pytest.mark.parametrize("scale,softcap", [(s, 0.0) for s in SCALES] + [(1.2 * 2.0 ** 40, 1e20), (1.2 * 2.0 ** 30, 1e16)])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_prompts(gpu_lib, D, scale, softcap):
    scale = float(np.float32(scale))
    for tokens, Hq, Hkv in ((300, 2, 1), (41, 1, 1), (29, 4, 2)):
        a, b, v = one_value_each(tokens, tokens, Hq, Hkv, D, 0)
        q, k = np.zeros((tokens, Hq, D)), np.zeros((tokens, Hkv, D))
        q[..., D - 3], k[..., D - 3] = a, b.T
        v = ref.bf16(v)
        o, lse = gpu_lib.prompt_attention(ref.bf16(q).cuda(), ref.bf16(k).cuda(), v.transpose(0, 1).cuda(),
                                          starts_of([tokens]), scale=scale, softcap=softcap, return_lse=True)
        hold_to_the_largest(o, lse, a, b, ref.f64(v), scale, softcap)


@pytest.mark.parametrize("scale,softcap", [(s, 0.0) for s in SCALES] + [(1.2 * 2.0 ** 40, 1e20)])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("fp8", [False, True])
def test_chunks(gpu_lib, fp8, D, scale, softcap):
    scale, page = float(np.float32(scale)), 16
    for tokens, keys, Hq, Hkv in ((3, 500, 4, 2), (41, 300, 1, 1), (150, 410, 2, 1)):
        a, b, v = one_value_each(tokens, keys, Hq, Hkv, D, 1)
        pages = -(-keys // page)

        def paged(x, fill):  # [Hkv, keys, ..] as pages in order
            out = torch.full((Hkv, pages * page, *x.shape[2:]), fill, dtype=x.dtype)
            out[:, :keys] = x
            return out.view(Hkv, pages, page, *x.shape[2:]).transpose(0, 1).contiguous().cuda()

        q = np.zeros((tokens, Hq, D))
        q[..., D - 3] = a
        if fp8:  # codes of 1 with the keys' values as scales
            k = torch.zeros(Hkv, keys, D, dtype=torch.uint8)
            k[..., D - 3] = 0x38
            s = torch.from_numpy(np.abs(v).max(-1).astype(np.float32) / np.float32(448))
            codes = torch.from_numpy(ref.e4m3_codes_f32(v.astype(np.float32), s.numpy()))
            v = ref.e4m3_values(codes) * ref.f64(s)[..., None]
            cache = [paged(k, 0x7F), paged(codes, 0x7F), paged(torch.from_numpy(b.astype(np.float32)), float("nan")),
                     paged(s, float("nan"))]
        else:
            k = np.zeros((Hkv, keys, D))
            k[..., D - 3] = b
            v = ref.f64(ref.bf16(v))
            cache = [paged(ref.bf16(k), float("nan")), paged(ref.bf16(v), float("nan"))]
        call = gpu_lib.paged_chunk_attention_fp8 if fp8 else gpu_lib.paged_chunk_attention
        o, lse = call(ref.bf16(q).cuda(), *cache, torch.arange(pages, dtype=torch.int32, device="cuda")[None],
                      torch.tensor([keys], dtype=torch.int32, device="cuda"), starts_of([tokens]), scale=scale,
                      softcap=softcap, return_lse=True)
        hold_to_the_largest(o, lse, a, b, v, scale, softcap)
