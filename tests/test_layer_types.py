"""Which float8 tensors the decoder-layer calls take for bytes: e4m3 ones for codes,
UE8M0 ones for scale bytes, and neither for the other."""
from __future__ import annotations

import pytest
import torch

import sparse_gemm_linears_amd as sgl

CODES, SCALES = torch.float8_e4m3fn, torch.float8_e8m0fnu


def test_cache_codes():
    q = torch.zeros(1, 1, 64, dtype=torch.bfloat16)
    qkv = torch.zeros(1, 192, dtype=torch.bfloat16)
    cache = torch.zeros(1, 1, 16, 64, dtype=torch.uint8)
    for call in (lambda k: sgl.paged_decode_attention_fp8(q, k, k, None, None, None, None),
                 lambda k: sgl.kv_rope_append_fp8(qkv, None, None, None, k, k, None, None)):
        for kind in (torch.uint8, CODES):  # past the type, refused because they are host tensors
            with pytest.raises(ValueError, match="device tensor"):
                call(cache.view(kind))
        for kind in (SCALES, torch.int8, torch.float8_e5m2):
            with pytest.raises(TypeError, match="k_cache"):
                call(cache.view(kind))


@pytest.mark.gpu
def test_norm_outputs(gpu_lib):
    x = torch.randn(3, 256, device="cuda").bfloat16()
    w = torch.ones(256, device="cuda", dtype=torch.bfloat16)
    want = gpu_lib.fp8_add_rmsnorm_ue8m0(x, w)
    for code, scale in ((torch.uint8, torch.uint8), (CODES, SCALES)):
        q = torch.empty(3, 256, dtype=torch.uint8, device="cuda").view(code)
        e = torch.empty(3, 2, dtype=torch.uint8, device="cuda").view(scale)
        got = gpu_lib.fp8_add_rmsnorm_ue8m0(x, w, q=q, e=e)
        assert got[2] is q and got[3] is e
        assert torch.equal(q.view(torch.uint8), want[2]) and torch.equal(e.view(torch.uint8), want[3])
    q, e = (torch.empty(3, n, dtype=torch.uint8, device="cuda") for n in (256, 2))
    with pytest.raises(TypeError, match="q"):
        gpu_lib.fp8_add_rmsnorm_ue8m0(x, w, q=q.view(SCALES), e=e)
    with pytest.raises(TypeError, match="scales"):
        gpu_lib.fp8_add_rmsnorm_ue8m0(x, w, q=q, e=e.view(CODES))
    with pytest.raises(TypeError, match="scales"):
        gpu_lib.fp8_add_rmsnorm(x, w, q=q, s=e)


@pytest.mark.gpu
def test_cache_of_codes_as_float8(gpu_lib):
    """A cache held as float8_e4m3fn tensors gives what the same bytes as uint8 give."""
    qkv = torch.randn(5, 3 * 64, device="cuda").bfloat16()
    positions, slots = torch.arange(5, dtype=torch.int32, device="cuda"), torch.arange(5, device="cuda")
    angle = torch.rand(8, 32, device="cuda")
    table = torch.cat([angle.cos(), angle.sin()], -1)
    pages = torch.zeros(1, 1, dtype=torch.int32, device="cuda")
    lens = torch.tensor([5], dtype=torch.int32, device="cuda")
    got = []
    for kind in (torch.uint8, CODES):
        k, v = (torch.zeros(1, 1, 16, 64, dtype=torch.uint8, device="cuda").view(kind) for _ in range(2))
        ks, vs = (torch.zeros(1, 1, 16, device="cuda") for _ in range(2))
        q = gpu_lib.kv_rope_append_fp8(qkv, positions, slots, table, k, v, ks, vs)
        got.append([q, k.view(torch.uint8), v.view(torch.uint8),
                    gpu_lib.paged_decode_attention_fp8(q[4:], k, v, ks, vs, pages, lens)])
    for a, b in zip(*got):
        assert torch.equal(a, b)
