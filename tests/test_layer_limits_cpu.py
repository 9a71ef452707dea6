"""The limits and alignments that fp8lin.h states for the decoder-layer calls: the last
allowed number passes every check (and stops at the device), the next one is refused."""
from __future__ import annotations

import ctypes

import pytest
import torch

import sparse_gemm_linears_amd as sgl

pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="allowed numbers would launch")
A, B, C, D, E, F, G, H, J = (i << 52 for i in range(1, 10))  # fake, farther apart than the largest cache
SHAPE, ALIGN, DEVICE = sgl.FP8L_ERR_SHAPE, sgl.FP8L_ERR_ALIGN, sgl.FP8L_ERR_DEVICE


def P(v):
    return ctypes.c_void_p(v) if v else None


def norm(x=A, res=B, w=C, M=4, K=256, h=D, y=E, q=F, s=G):
    return sgl.load_library().fp8_add_rmsnorm(P(x), P(res), P(w), 1e-5, M, K, P(h), P(y), P(q), P(s), None)


def append(pos=B, slots=C, T=4, Hq=8, Hkv=2, D_=128, rot=128, max_pos=64, pages=8, page=16):
    return sgl.load_library().kv_rope_append(P(A), P(pos), P(slots), P(D), T, Hq, Hkv, D_, rot, 0, max_pos, pages, page,
                                             P(E), P(F), P(G), None)


def attend(table=D, lens=E, lse=G, batch=3, Hq=8, Hkv=2, D_=128, pages=8, page=16, max_pages=4, max_len=64, window=0):
    return sgl.load_library().paged_decode_attention(P(A), P(B), P(C), P(table), P(lens), batch, Hq, Hkv, D_, pages, page,
                                                     max_pages, max_len, 0.1, 0.0, window, P(F), P(lse), None)


@pytest.mark.parametrize("call,last,after", [
    (norm, dict(M=1 << 24, K=128), dict(M=(1 << 24) + 1, K=128)),
    (norm, dict(M=1 << 12, K=1 << 24), dict(M=(1 << 12) + 1, K=1 << 24)),
    (norm, dict(M=1, K=1 << 24), dict(M=1, K=(1 << 24) + 128)),
    (append, dict(T=1 << 24, Hq=8), dict(T=(1 << 24) + 1, Hq=8)),
    (append, dict(T=1 << 21, Hq=252), dict(T=(1 << 21) + 1, Hq=252)),  # of 256 heads of 128: 2^36 values
    (append, dict(max_pos=1 << 24), dict(max_pos=(1 << 24) + 1)),
    (append, dict(max_pos=1), dict(max_pos=0)),
    (append, dict(rot=0, max_pos=0), dict(rot=0, max_pos=-1)),
    (append, dict(Hq=1024, Hkv=1024), dict(Hq=1025, Hkv=1024)),
    (append, dict(page=65536), dict(page=65536 + 16)),
    (append, dict(page=16), dict(page=8)),
    (append, dict(pages=(1 << 27) - 1, Hkv=1), dict(pages=1 << 27, Hkv=1)),  # slots below 2^31
    (append, dict(pages=1 << 22, Hkv=64, D_=256), dict(pages=(1 << 22) + 1, Hkv=64, D_=256)),  # 2^40 values
    (attend, dict(batch=65535), dict(batch=65536)),
    (attend, dict(max_pages=1 << 26, max_len=1 << 30), dict(max_pages=(1 << 26) + 1)),
    (attend, dict(max_len=64), dict(max_len=65)),
    (attend, dict(max_len=0), dict(max_len=-1)),
    (attend, dict(max_pages=1, max_len=0), dict(max_pages=0, max_len=0)),
    (attend, dict(window=(1 << 63) - 1), dict(window=-1)),
    (attend, dict(Hq=1024, Hkv=1), dict(Hq=1025, Hkv=1)),
])
def test_limits(call, last, after):
    assert call(**last) == DEVICE and call(**after) == SHAPE


@pytest.mark.parametrize("call,name,base,step", [(append, "pos", B, 4), (append, "slots", C, 8), (attend, "table", D, 4),
                                                 (attend, "lens", E, 4), (attend, "lse", G, 4)])
def test_alignments(call, name, base, step):
    assert call(**{name: base + step}) == DEVICE and call(**{name: base + step // 2}) == ALIGN


def test_status_text_of_alignment():
    assert "as stated with the call" in sgl.status_str(ALIGN)
