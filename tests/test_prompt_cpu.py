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
