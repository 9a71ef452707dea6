"""Refusals of the decoder-layer calls, checked without a GPU: every invalid
argument gives its documented status before any HIP call, and the binding
rejects wrong types, shapes and host tensors."""
from __future__ import annotations

import ctypes

import pytest
import torch

import sparse_gemm_linears_amd as sgl

A, B, C, D, E, F, G, H, J = (i << 34 for i in range(1, 10))  # fake, far apart and 16-byte aligned


def P(v):
    return ctypes.c_void_p(v) if v else None


@pytest.fixture(scope="module")
def lib():
    return sgl.load_library()


@pytest.mark.parametrize("name", ["fp8_add_rmsnorm", "fp8_add_rmsnorm_ue8m0"])
def test_norm_refusals(lib, name):
    def f(x=A, res=B, w=C, eps=1e-5, M=4, K=256, h=D, y=E, q=F, s=G):
        return getattr(lib, name)(P(x), P(res), P(w), eps, M, K, P(h), P(y), P(q), P(s), None)

    for bad in (dict(K=100), dict(K=0), dict(M=-1), dict(K=1 << 25), dict(M=1 << 25), dict(M=1 << 24, K=1 << 24),
                dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf"))):
        assert f(**bad) == sgl.FP8L_ERR_SHAPE, bad
    for bad in (dict(x=0), dict(w=0), dict(res=0), dict(h=0), dict(q=0), dict(s=0), dict(y=0, q=0, s=0)):
        assert f(**bad) == sgl.FP8L_ERR_NULL, bad
    for bad in (dict(x=A + 8), dict(w=C + 2), dict(q=F + 8), dict(s=G + 4), dict(h=D + 8), dict(y=E + 8)):
        assert f(**bad) == sgl.FP8L_ERR_ALIGN, bad
    for bad in (dict(h=A), dict(y=B + 16), dict(q=C), dict(q=D + 1024), dict(s=F + 16), dict(h=B + 16)):
        assert f(**bad) == sgl.FP8L_ERR_ALIAS, bad
    assert f(M=0, x=0, res=0, w=0, h=0, y=0, q=0, s=0) == sgl.FP8L_OK
    if not torch.cuda.is_available():
        assert f() == sgl.FP8L_ERR_DEVICE
        assert f(h=B) == sgl.FP8L_ERR_DEVICE  # in place is allowed
        assert f(res=0, h=0, y=0) == sgl.FP8L_ERR_DEVICE
        assert f(q=0, s=0) == sgl.FP8L_ERR_DEVICE


@pytest.mark.parametrize("fp8", [False, True])
def test_append_refusals(lib, fp8):
    def f(qkv=A, pos=B, slots=C, cs=D, T=4, Hq=8, Hkv=2, D_=128, rot=128, inter=0, max_pos=64, pages=8, page=16, q=E,
          k=F, v=G, ks=H, vs=J):
        args = [P(qkv), P(pos), P(slots), P(cs), T, Hq, Hkv, D_, rot, inter, max_pos, pages, page, P(q), P(k), P(v)]
        if fp8:
            return lib.kv_rope_append_fp8(*args, P(ks), P(vs), None)
        return lib.kv_rope_append(*args, None)

    big = 1 << 62
    for bad in (dict(T=-1), dict(T=1 << 25), dict(Hq=0), dict(Hkv=0), dict(Hq=2000), dict(D_=96), dict(D_=0),
                dict(rot=-16), dict(rot=144), dict(rot=8), dict(max_pos=0), dict(pages=0), dict(page=0),
                dict(page=24), dict(page=1 << 17), dict(pages=1 << 30), dict(pages=big), dict(T=big),
                dict(max_pos=big)):
        assert f(**bad) == sgl.FP8L_ERR_SHAPE, bad
    for bad in (dict(qkv=0), dict(pos=0), dict(slots=0), dict(cs=0), dict(q=0), dict(k=0), dict(v=0)) + (
            (dict(ks=0), dict(vs=0)) if fp8 else ()):
        assert f(**bad) == sgl.FP8L_ERR_NULL, bad
    for bad in (dict(qkv=A + 8), dict(pos=B + 2), dict(slots=C + 4), dict(cs=D + 8), dict(q=E + 2), dict(k=F + 8)):
        assert f(**bad) == sgl.FP8L_ERR_ALIGN, bad
    for bad in (dict(q=A), dict(k=A + 16), dict(v=F + 4096), dict(q=C), dict(k=D)):
        assert f(**bad) == sgl.FP8L_ERR_ALIAS, bad
    if fp8:
        assert f(ks=H, vs=H + 16) == sgl.FP8L_ERR_ALIAS
    assert f(T=0, qkv=0, pos=0, slots=0, cs=0, q=0, k=0, v=0) == sgl.FP8L_OK
    if not torch.cuda.is_available():
        assert f() == sgl.FP8L_ERR_DEVICE
        assert f(rot=0, pos=0, cs=0) == sgl.FP8L_ERR_DEVICE


@pytest.mark.parametrize("fp8", [False, True])
def test_attention_refusals(lib, fp8):
    def f(q=A, k=B, v=C, ks=H, vs=J, table=D, lens=E, batch=3, Hq=8, Hkv=2, D_=128, pages=8, page=16, max_pages=4,
          max_len=64, scale=0.1, cap=0.0, window=0, o=F, lse=G):
        tail = [P(table), P(lens), batch, Hq, Hkv, D_, pages, page, max_pages, max_len, scale, cap, window, P(o),
                P(lse), None]
        if fp8:
            return lib.paged_decode_attention_fp8(P(q), P(k), P(v), P(ks), P(vs), *tail)
        return lib.paged_decode_attention(P(q), P(k), P(v), *tail)

    big = 1 << 62
    for bad in (dict(batch=-1), dict(batch=65536), dict(Hq=9), dict(Hq=0), dict(Hkv=0), dict(D_=32), dict(page=20),
                dict(pages=0), dict(max_pages=0), dict(max_len=65), dict(max_len=-1), dict(window=-1),
                dict(scale=float("nan")), dict(scale=float("inf")), dict(cap=-1.0), dict(cap=float("inf")),
                dict(cap=float("nan")), dict(pages=big), dict(max_pages=big), dict(max_len=big), dict(page=big)):
        assert f(**bad) == sgl.FP8L_ERR_SHAPE, bad
    for bad in (dict(q=0), dict(k=0), dict(v=0), dict(table=0), dict(lens=0), dict(o=0)) + (
            (dict(ks=0), dict(vs=0)) if fp8 else ()):
        assert f(**bad) == sgl.FP8L_ERR_NULL, bad
    for bad in (dict(q=A + 8), dict(k=B + 2), dict(table=D + 1), dict(lens=E + 2), dict(o=F + 8), dict(lse=G + 2)):
        assert f(**bad) == sgl.FP8L_ERR_ALIGN, bad
    for bad in (dict(o=A), dict(o=B + 16), dict(o=C), dict(lse=E), dict(lse=F + 4), dict(o=D)):
        assert f(**bad) == sgl.FP8L_ERR_ALIAS, bad
    assert f(batch=0, q=0, k=0, v=0, table=0, lens=0, o=0, lse=0) == sgl.FP8L_OK
    if not torch.cuda.is_available():
        assert f() == sgl.FP8L_ERR_DEVICE
        assert f(lse=0, window=big) == sgl.FP8L_ERR_DEVICE


def test_binding_refusals():
    x, w = torch.zeros(2, 128, dtype=torch.bfloat16), torch.ones(128, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        sgl.fp8_add_rmsnorm(x, w)  # host tensors
    with pytest.raises(TypeError):
        sgl.fp8_add_rmsnorm(x.float(), w)
    cache = torch.zeros(1, 1, 16, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        sgl.kv_rope_append(x, torch.zeros(2, dtype=torch.int32), torch.zeros(2, dtype=torch.int64),
                           torch.zeros(4, 64), cache, cache)
    with pytest.raises(TypeError):
        sgl.paged_decode_attention(x, cache.float(), cache, None, None)
