"""Refusals of the calls for prompts and chunks, checked without a GPU: every invalid
argument gives its documented status before any HIP call."""
from __future__ import annotations

import ctypes

import pytest
import torch

import sparse_gemm_linears_amd as sgl

A, B, C, D, E, F, G, H, J, K, L, M = (i << 44 for i in range(1, 13))  # fake, far apart and 16-byte aligned


def P(v):
    return ctypes.c_void_p(v) if v else None


@pytest.fixture(scope="module")
def lib():
    return sgl.load_library()


@pytest.mark.parametrize("fp8", [False, True])
def test_norm_append_refusals(lib, fp8):
    def f(qkv=A, qw=K, kw=L, eps=1e-6, pos=B, slots=C, cs=D, T=4, Hq=8, Hkv=2, D_=128, rot=128, inter=0, max_pos=64,
          pages=8, page=16, q=E, ko=M, k=F, v=G, ks=H, vs=J):
        args = [P(qkv), P(qw), P(kw), eps, P(pos), P(slots), P(cs), T, Hq, Hkv, D_, rot, inter, max_pos, pages, page,
                P(q), P(ko), P(k), P(v)]
        if fp8:
            return lib.kv_norm_rope_append_fp8(*args, P(ks), P(vs), None)
        return lib.kv_norm_rope_append(*args, None)

    big = 1 << 62
    for bad in (dict(T=-1), dict(T=1 << 25), dict(Hq=0), dict(Hkv=0), dict(Hq=2000), dict(D_=96), dict(rot=144),
                dict(rot=8), dict(max_pos=0), dict(pages=0), dict(page=24), dict(pages=big), dict(T=big),
                dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf"))):
        assert f(**bad) == sgl.FP8L_ERR_SHAPE, bad
    for bad in (dict(qkv=0), dict(pos=0), dict(slots=0), dict(cs=0), dict(q=0), dict(k=0), dict(v=0)) + (
            (dict(ks=0), dict(vs=0)) if fp8 else ()):
        assert f(**bad) == sgl.FP8L_ERR_NULL, bad
    for bad in (dict(qkv=A + 8), dict(qw=K + 8), dict(kw=L + 2), dict(ko=M + 8), dict(pos=B + 2), dict(slots=C + 4)):
        assert f(**bad) == sgl.FP8L_ERR_ALIGN, bad
    for bad in (dict(q=A), dict(ko=A + 16), dict(ko=E), dict(k=K), dict(v=L), dict(ko=F + 4096), dict(q=K), dict(qw=M)):
        assert f(**bad) == sgl.FP8L_ERR_ALIAS, bad
    assert f(T=0, qkv=0, pos=0, slots=0, cs=0, q=0, ko=0, k=0, v=0) == sgl.FP8L_OK
    if not torch.cuda.is_available():
        for fine in (dict(), dict(qw=0), dict(kw=0), dict(ko=0), dict(qw=0, kw=0, ko=0), dict(eps=0.0), dict(kw=K)):
            assert f(**fine) == sgl.FP8L_ERR_DEVICE, fine


def test_prompt_refusals(lib):
    def f(q=A, k=B, v=C, starts=D, batch=3, T=64, Hq=8, Hkv=2, D_=128, strides=(1024, 128, 256, 128, 256, 128), scale=0.1,
          cap=0.0, window=0, causal=1, o=E, lse=F):
        return lib.prompt_attention(P(q), P(k), P(v), P(starts), batch, T, Hq, Hkv, D_, *strides, scale, cap, window, causal,
                                    P(o), P(lse), None)

    big = 1 << 62
    for bad in (dict(batch=-1), dict(batch=65536), dict(T=-1), dict(T=(1 << 24) + 1), dict(T=1 << 24, Hq=1024), dict(T=big),
                dict(Hq=9), dict(Hq=0), dict(Hkv=0), dict(Hq=1026), dict(D_=32), dict(D_=96), dict(window=-1),
                dict(window=8, causal=0), dict(scale=float("nan")), dict(scale=float("inf")), dict(scale=2.0 ** 101),
                dict(scale=-2.0 ** 101), dict(cap=-1.0), dict(cap=float("inf")), dict(cap=float("nan"))):
        assert f(**bad) == sgl.FP8L_ERR_SHAPE, bad
    for i in range(6):
        for stride in (-8, 4, 1, (1 << (36 if i % 2 else 24)) + 8, big):
            strides = [1024, 128, 256, 128, 256, 128]
            strides[i] = stride
            assert f(strides=strides) == sgl.FP8L_ERR_SHAPE, strides
    for bad in (dict(q=0), dict(k=0), dict(v=0), dict(starts=0), dict(o=0)):
        assert f(**bad) == sgl.FP8L_ERR_NULL, bad
    for bad in (dict(q=A + 8), dict(k=B + 2), dict(v=C + 8), dict(o=E + 8), dict(starts=D + 2), dict(lse=F + 2)):
        assert f(**bad) == sgl.FP8L_ERR_ALIGN, bad
    # the last value of a strided input counts
    for bad in (dict(o=A), dict(o=B), dict(o=C + 256), dict(o=D), dict(lse=E + 4), dict(lse=D + 4),
                dict(o=A + (1 << 30), strides=(1 << 24, 128, 256, 128, 256, 128))):
        assert f(**bad) == sgl.FP8L_ERR_ALIAS, bad
    assert f(batch=0, q=0, k=0, v=0, starts=0, o=0, lse=0) == sgl.FP8L_OK
    assert f(T=0, q=0, k=0, v=0, starts=0, o=0, lse=0) == sgl.FP8L_OK
    if not torch.cuda.is_available():
        for fine in (dict(), dict(lse=0), dict(window=big), dict(causal=0), dict(scale=0.0), dict(scale=-(2.0 ** 100)),
                     dict(strides=(0,) * 6), dict(k=A, v=A), dict(Hq=1024, Hkv=1, strides=(8,) * 6),
                     dict(T=1 << 24, Hq=64, D_=64, o=M), dict(batch=65535),
                     dict(strides=(1 << 24, 1 << 36) * 3, Hq=2, o=M << 4, lse=L << 4)):
            assert f(**fine) == sgl.FP8L_ERR_DEVICE, fine


@pytest.mark.parametrize("fp8", [False, True])
def test_chunk_refusals(lib, fp8):
    def f(q=A, k=B, v=C, ks=H, vs=J, table=D, lens=E, starts=K, batch=3, T=64, Hq=8, Hkv=2, D_=128, pages=8, page=16,
          max_pages=4, max_len=64, scale=0.1, cap=0.0, window=0, o=F, lse=G):
        tail = [P(table), P(lens), P(starts), batch, T, Hq, Hkv, D_, pages, page, max_pages, max_len, scale, cap, window,
                P(o), P(lse), None]
        if fp8:
            return lib.paged_chunk_attention_fp8(P(q), P(k), P(v), P(ks), P(vs), *tail)
        return lib.paged_chunk_attention(P(q), P(k), P(v), *tail)

    big = 1 << 62
    for bad in (dict(batch=-1), dict(batch=65536), dict(T=-1), dict(T=(1 << 24) + 1), dict(T=big), dict(Hq=9), dict(Hq=0),
                dict(Hkv=0), dict(D_=32), dict(page=20), dict(pages=0), dict(max_pages=0), dict(max_len=65),
                dict(max_len=-1), dict(window=-1), dict(scale=float("nan")), dict(scale=2.0 ** 101), dict(cap=-1.0),
                dict(cap=float("inf")), dict(pages=big), dict(max_pages=big), dict(max_len=big), dict(page=big)):
        assert f(**bad) == sgl.FP8L_ERR_SHAPE, bad
    for bad in (dict(q=0), dict(k=0), dict(v=0), dict(table=0), dict(lens=0), dict(starts=0), dict(o=0)) + (
            (dict(ks=0), dict(vs=0)) if fp8 else ()):
        assert f(**bad) == sgl.FP8L_ERR_NULL, bad
    for bad in (dict(q=A + 8), dict(k=B + 2), dict(table=D + 1), dict(lens=E + 2), dict(starts=K + 2), dict(o=F + 8),
                dict(lse=G + 2)):
        assert f(**bad) == sgl.FP8L_ERR_ALIGN, bad
    for bad in (dict(o=A), dict(o=B + 16), dict(o=C), dict(lse=E), dict(lse=F + 4), dict(o=D), dict(o=K), dict(lse=K + 12)):
        assert f(**bad) == sgl.FP8L_ERR_ALIAS, bad
    assert f(batch=0, q=0, k=0, v=0, table=0, lens=0, starts=0, o=0, lse=0) == sgl.FP8L_OK
    assert f(T=0, q=0, k=0, v=0, table=0, lens=0, starts=0, o=0, lse=0) == sgl.FP8L_OK
    if not torch.cuda.is_available():
        for fine in (dict(), dict(lse=0, window=big), dict(lse=K + 16), dict(T=1 << 24, Hq=64, D_=64), dict(max_len=0)):
            assert f(**fine) == sgl.FP8L_ERR_DEVICE, fine


def test_binding_takes_device_tensors_only():
    x = torch.zeros(2, 4, 64, dtype=torch.bfloat16)
    starts = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="device"):
        sgl.prompt_attention(x, x, x, starts)
    with pytest.raises(TypeError):
        sgl.prompt_attention(x.float(), x, x, starts)
    with pytest.raises(TypeError):
        sgl.prompt_attention(None, x, x, starts)
    cache = torch.zeros(1, 1, 16, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="device"):
        sgl.paged_chunk_attention(x, cache, cache, starts, starts, starts)
    with pytest.raises(ValueError, match="device"):
        sgl.kv_norm_rope_append(x.view(2, 256), None, None, starts, starts, x, cache, cache)
