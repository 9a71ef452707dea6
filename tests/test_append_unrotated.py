"""The append without rotation (rot = 0): no table is read, so one without rows is as good as any."""
from __future__ import annotations

import ctypes

import pytest
import torch

import sparse_gemm_linears_amd as sgl

P = ctypes.c_void_p
QKV, SLOTS, Q, K, V, KS, VS = (P(i << 34) for i in range(1, 8))  # far apart and 16-byte aligned


@pytest.mark.parametrize("fp8", [False, True])
def test_table_sizes(fp8):
    lib = sgl.load_library()

    def call(T=0, rot=0, max_pos=0, table=None, positions=None):
        args = [QKV, positions, SLOTS, table, T, 8, 2, 128, rot, 0, max_pos, 8, 16, Q, K, V]
        return lib.kv_rope_append_fp8(*args, KS, VS, None) if fp8 else lib.kv_rope_append(*args, None)

    assert call() == sgl.FP8L_OK and call(max_pos=7) == sgl.FP8L_OK
    assert call(max_pos=-1) == sgl.FP8L_ERR_SHAPE
    assert call(rot=16, max_pos=0) == sgl.FP8L_ERR_SHAPE
    if not torch.cuda.is_available():
        assert call(T=4) == sgl.FP8L_ERR_DEVICE


@pytest.mark.gpu
@pytest.mark.parametrize("rows", [0, 1, 5])
@pytest.mark.parametrize("fp8", [False, True])
def test_append_copies(gpu_lib, fp8, rows):
    T, hq, hkv, d = 5, 4, 2, 64
    qkv = torch.randn(T, (hq + 2 * hkv) * d, device="cuda").bfloat16()
    kind = torch.uint8 if fp8 else torch.bfloat16
    k, v = (torch.zeros(1, hkv, 16, d, dtype=kind, device="cuda") for _ in range(2))
    scales = [torch.zeros(1, hkv, 16, device="cuda") for _ in range(2)] if fp8 else []
    positions = torch.full((T,), 3, dtype=torch.int32, device="cuda")
    call = gpu_lib.kv_rope_append_fp8 if fp8 else gpu_lib.kv_rope_append
    q = call(qkv, positions, torch.arange(T, device="cuda"), torch.empty(rows, 0, device="cuda"), k, v, *scales)
    heads = qkv.view(T, hq + 2 * hkv, d)
    assert torch.equal(q, heads[:, :hq])
    for i, cache in enumerate((k, v)):
        want = heads[:, hq + i * hkv : hq + (i + 1) * hkv].transpose(0, 1)
        if not fp8:
            assert torch.equal(cache[0, :, :T], want)
            continue
        # the scale is amax / 448 in fp32 (a division of the GPU's may be one step off), a code half a step
        amax = want.float().abs().amax(-1)
        s = scales[i][0, :, :T]
        assert ((s - amax / 448).abs() <= 2.0 ** -22 * s).all()
        got = cache[0, :, :T].contiguous().view(torch.float8_e4m3fn).float() * s[..., None]
        assert ((got - want.float()).abs() <= torch.maximum(2.0 ** -4 * want.float().abs(), 2.0 ** -10 * s[..., None])
                * (1 + 2.0 ** -10)).all()
