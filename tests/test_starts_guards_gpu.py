"""Starts that are out of order or outside the rows: nothing but the rows of o and lse is written.  Both lie between
guards of several blocks of rows; what the rows themselves hold is unspecified."""
from __future__ import annotations

import pytest
import torch

import layer_ref as ref
from test_chunk_gpu import shared_pages
from test_layer_gpu import gen
from test_prompt_gpu import inputs, starts_of

pytestmark = pytest.mark.gpu

GUARD = 400  # tokens: more than three blocks of 128 rows on either side


class Guarded:
    """o and lse of T tokens, in the middle of larger buffers."""

    def __init__(self, T, Hq, D):
        self.T = T
        self.o_all = torch.full((T + 2 * GUARD, Hq, D), 7.0, dtype=torch.bfloat16, device="cuda")
        self.lse_all = torch.full((T + 2 * GUARD, Hq), 7.0, device="cuda")
        self.o, self.lse = self.o_all[GUARD : GUARD + T], self.lse_all[GUARD : GUARD + T]

    def hold(self, what):
        torch.cuda.synchronize()
        for t in (self.o_all, self.lse_all):
            assert (t[:GUARD] == 7).all() and (t[GUARD + self.T :] == 7).all(), what


def bad_starts(T, B):
    """Of B sequences over T rows."""
    far = 1 << 30
    return [[T - i * T // B for i in range(B + 1)], [0 if b % 2 else T for b in range(B + 1)],
            [0 if b % 2 else far for b in range(B + 1)], [-(1 << 31)] * B + [(1 << 31) - 1], [far] * (B + 1),
            [T // 2] + [0] * (B - 1) + [T], [-5] + [(b * 7919) % (2 * T) for b in range(B)]]


@pytest.mark.parametrize("T,B,Hq,Hkv,D", [(12, 3, 2, 1, 64), (300, 3, 8, 2, 128), (300, 70, 4, 2, 64), (130, 2, 2, 1, 256)])
def test_prompts(gpu_lib, T, B, Hq, Hkv, D):
    q, k, v = (t.cuda() for t in inputs([T], Hq, Hkv, D))
    for starts in bad_starts(T, B):
        for causal in (True, False):
            out = Guarded(T, Hq, D)
            gpu_lib.prompt_attention(q, k, v, torch.tensor(starts, dtype=torch.int32, device="cuda"), causal=causal,
                                     o=out.o, lse=out.lse, return_lse=True)
            out.hold(starts[:8])


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("T,B,group,Hkv,D", [(12, 3, 2, 1, 64), (300, 3, 4, 2, 128), (300, 100, 8, 1, 64), (300, 260, 2, 1, 64),
                                             (40, 1, 4, 1, 128), (130, 2, 2, 1, 256)])
def test_chunks(gpu_lib, T, B, group, Hkv, D, fp8):
    """Over caches long enough that sequences are divided."""
    cache, row, _ = shared_pages(D, Hkv, 2000, 16, fp8, 3)
    q = ref.bf16(gen("guards", T, B, D).standard_normal((T, Hkv * group, D))).cuda()
    call = gpu_lib.paged_chunk_attention_fp8 if fp8 else gpu_lib.paged_chunk_attention
    table = row.expand(B, -1).contiguous()
    for lens in (torch.full((B,), 2000), 1 + 50 * torch.arange(B) % 2000):
        for starts in bad_starts(T, B):
            out = Guarded(T, Hkv * group, D)
            call(q, *cache, table, lens.int().cuda(), torch.tensor(starts, dtype=torch.int32, device="cuda"), o=out.o,
                 lse=out.lse, return_lse=True)
            out.hold(starts[:8])
    # and the call as it should be writes every row
    new = [T // B + (b < T % B) for b in range(B)]
    out = Guarded(T, Hkv * group, D)
    call(q, *cache, table, torch.full((B,), 2000, dtype=torch.int32, device="cuda"), starts_of(new), o=out.o,
         lse=out.lse, return_lse=True)
    out.hold("in order")
    assert not (out.lse == 7).any()
