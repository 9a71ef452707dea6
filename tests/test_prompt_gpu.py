"""prompt_attention against the 64-bit reference (tolerances in prompt_ref.py)."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import layer_ref as ref
from prompt_ref import Check, heads
from test_graph_gpu import replay_equals_eager
from test_layer_gpu import gen

pytestmark = pytest.mark.gpu


def starts_of(lens, first=0):
    return torch.tensor(np.concatenate([[0], np.cumsum(lens)]) + first, dtype=torch.int32, device="cuda")


def inputs(lens, Hq, Hkv, D, sharp=1.5, extra=0):
    r = gen("prompt", sum(lens), len(lens), Hq, Hkv, D)
    T = sum(lens) + extra
    return [ref.bf16(f * r.standard_normal((T, n, D))) for f, n in ((sharp, Hq), (1.0, Hkv), (1.0, Hkv))]


def prompt_case(lib, lens, Hq, Hkv, D, causal=True, window=0, softcap=0.0, scale=None, sharp=1.5, views=None):
    q, k, v = inputs(lens, Hq, Hkv, D, sharp)
    dev = [t.cuda() for t in (q, k, v)] if views is None else views(q, k, v)
    kw = dict(causal=causal, window=window, softcap=softcap, scale=scale)
    print(f"prompt lens={lens[:8]} Hq={Hq} Hkv={Hkv} D={D} {kw}", flush=True)
    starts = starts_of(lens)
    o, lse = lib.prompt_attention(*dev, starts, **kw, return_lse=True)
    again = lib.prompt_attention(*dev, starts, **kw)
    torch.cuda.synchronize()
    assert torch.equal(o, again)  # deterministic, and the same without lse
    check, at = Check(D ** -0.5 if scale is None else scale, softcap), 0
    for i, n in enumerate(lens):
        rows = slice(at, at + n)
        if n:
            check.sequence(o[rows], lse[rows], ref.f64(q[rows]), heads(k[rows]), heads(v[rows]), 0, window, causal,
                           f"of prompt {i}, length {n}")
        at += n
    check.done()
    return o, lse


EDGES = [1, 0, 2, 3, 7, 8, 9, 15, 16, 17, 31, 32, 33, 63, 64, 65, 96, 127, 128, 129, 200, 0]


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("Hq,Hkv,D", [(8, 2, 128), (7, 1, 64), (4, 2, 256), (3, 3, 128), (3, 3, 64), (2, 2, 256),
                                      (33, 1, 64), (16, 1, 128), (20, 4, 128), (70, 1, 256)])
def test_prompt_edges(gpu_lib, Hq, Hkv, D, causal):
    prompt_case(gpu_lib, EDGES, Hq, Hkv, D, causal)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("n", [1, 5, 16, 31, 64, 77, 300, 1023])
@pytest.mark.parametrize("Hq,Hkv,D", [(32, 8, 128), (6, 6, 64), (10, 1, 256)])
def test_one_prompt(gpu_lib, n, Hq, Hkv, D, causal):
    prompt_case(gpu_lib, [n], Hq, Hkv, D, causal)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("window,softcap", [(1, 0.0), (2, 0.0), (16, 0.0), (17, 30.0), (64, 0.0), (100, 0.0),
                                            (257, 5.0), (5000, 0.0), (0, 30.0), (1 << 40, 1.0)])
def test_window_and_cap(gpu_lib, window, softcap, D):
    prompt_case(gpu_lib, [700, 3, 129, 64, 1], 4, 2, D, window=window, softcap=softcap)


@pytest.mark.parametrize("softcap", [1e-40, 1e-3, 0.5, 300.0, 1e6, 1e30, 3e38])
def test_caps_of_any_size(gpu_lib, softcap):
    prompt_case(gpu_lib, [1, 40, 200], 6, 2, 64, softcap=softcap)


@pytest.mark.parametrize("scale", [0.0, -0.125, 1e-20, 1.0, 4.0])
def test_scales(gpu_lib, scale):
    """No scale, negative ones (the smallest product counts most), tiny and sharp ones."""
    prompt_case(gpu_lib, [5, 150, 70], 4, 2, 64, scale=scale)
    prompt_case(gpu_lib, [5, 150, 70], 4, 2, 128, scale=scale, softcap=20.0)


@pytest.mark.parametrize("lens,Hq,Hkv,D,window", [([4097], 4, 1, 128, 0), ([2500, 1700], 2, 2, 64, 0),
                                                  ([3001], 2, 1, 256, 0), ([4500], 4, 1, 128, 1000),
                                                  ([1, 4000, 1], 1, 1, 128, 0), ([3000, 10], 28, 4, 64, 0)])
def test_long(gpu_lib, lens, Hq, Hkv, D, window):
    prompt_case(gpu_lib, lens, Hq, Hkv, D, window=window)


def test_many_prompts(gpu_lib):
    """More prompts than a wave's lanes, twice over in the search; empty ones among them."""
    r = gen("many")
    lens = [int(x) for x in np.where(r.random(5000) < 0.3, 0, r.integers(1, 4, 5000))]
    prompt_case(gpu_lib, lens, 2, 1, 64)


def test_many_prompts_of_many_heads(gpu_lib):
    lens = [int(x) for x in gen("heads").integers(0, 3, 130)]
    prompt_case(gpu_lib, lens, 256, 128, 64)
    prompt_case(gpu_lib, [40, 3], 1024, 1, 64)


def test_strided_views(gpu_lib):
    """Views of one projection, of padded rows, of heads in front of tokens, and heads repeated by a stride of 0."""
    lens, Hq, Hkv, D = [70, 1, 200], 8, 2, 128
    T = sum(lens)

    def projection(q, k, v):
        x = torch.cat([q, k, v], 1).reshape(T, -1).cuda()
        y = x.view(T, Hq + 2 * Hkv, D)
        return y[:, :Hq], y[:, Hq : Hq + Hkv], y[:, Hq + Hkv :]

    def padded(q, k, v):
        out = []
        for t in (q, k, v):
            x = torch.full((T, t.shape[1] + 1, D + 8), float("nan"), dtype=torch.bfloat16, device="cuda")
            x[:, :-1, :D] = t.cuda()
            out.append(x[:, :-1, :D])
        return out

    def heads_first(q, k, v):
        return [t.transpose(0, 1).contiguous().cuda().transpose(0, 1) for t in (q, k, v)]

    want = prompt_case(gpu_lib, lens, Hq, Hkv, D)
    for views in (projection, padded, heads_first):
        got = prompt_case(gpu_lib, lens, Hq, Hkv, D, views=views)
        assert all(torch.equal(a, b) for a, b in zip(want, got)), views.__name__
    q, k, v = (t.cuda() for t in inputs(lens, Hq, 1, D))
    one = gpu_lib.prompt_attention(q, k.expand(T, 4, D), v.expand(T, 4, D), starts_of(lens))
    assert torch.equal(one, gpu_lib.prompt_attention(q, k.repeat(1, 4, 1), v.repeat(1, 4, 1), starts_of(lens)))
    ref_o = gpu_lib.prompt_attention(q, k, v, starts_of(lens))  # the same rows in another grouping
    assert ((ref_o.float() - one.float()).abs().max() < 2.0 ** -5).item()


def test_strides_past_32_bits(gpu_lib):
    """Tokens so far apart that their offsets do not fit 32 bits."""
    T, D = 2100, 64
    wide = torch.empty(T, 1 << 20, dtype=torch.bfloat16, device="cuda")  # 2^31 values and more
    q, k, v = (t.cuda() for t in inputs([T], 2, 1, D))
    views = []
    for i, t in enumerate((q, k, v)):
        at = wide[:, i << 10 : (i << 10) + t.shape[1] * D].view(T, t.shape[1], D)
        at.copy_(t)
        views.append(at)
    want = gpu_lib.prompt_attention(q, k, v, starts_of([T]))
    assert torch.equal(gpu_lib.prompt_attention(*views, starts_of([T])), want)


def test_prompts_of_falling_and_rising_lengths(gpu_lib):
    """Up to 64 prompts begin with their longest rows first, whatever their order."""
    lens = [int(x) for x in 2 ** gen("order").uniform(0, 9.5, 64)]
    for order in (sorted(lens), sorted(lens, reverse=True), lens, lens[:63] + [0], [0] * 63 + [130], lens + [7, 700]):
        prompt_case(gpu_lib, order, 4, 2, 64)


def test_rows_outside_every_prompt_stay(gpu_lib):
    lens, Hq, Hkv, D = [33, 0, 100], 4, 2, 64
    q, k, v = (t.cuda() for t in inputs(lens, Hq, Hkv, D, extra=30))
    T = sum(lens) + 30
    o = torch.full((T, Hq, D), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((T, Hq), 7.0, device="cuda")
    starts = starts_of(lens, 11)
    got = gpu_lib.prompt_attention(q, k, v, starts, o=o, lse=lse)
    assert got is o
    want = gpu_lib.prompt_attention(q[11:-19], k[11:-19], v[11:-19], starts_of(lens))
    assert torch.equal(o[11:-19], want)
    for t in (o, lse):
        assert (t[:11] == 7).all() and (t[-19:] == 7).all() and not (t[11:-19] == 7).any()


def test_hidden_values_do_not_reach_a_row(gpu_lib):
    """Infinities and NaN in keys and values after a row's place, before its window, or in another prompt."""
    n, Hq, Hkv = 150, 4, 2
    for D in (64, 128, 256):
        for window in (0, 40):
            q, k, v = (t.cuda() for t in inputs([n, 20], Hq, Hkv, D))
            starts = starts_of([n, 20])
            want, want_lse = gpu_lib.prompt_attention(q, k, v, starts, window=window, return_lse=True)
            for bad in (float("inf"), float("-inf"), float("nan")):
                for at, where in ((100, "v"), (100, "k"), (3, "v"), (129, "v")):
                    k2, v2 = k.clone(), v.clone()
                    (v2 if where == "v" else k2)[at, :, 5::7] = bad
                    o, lse = gpu_lib.prompt_attention(q, k2, v2, starts, window=window, return_lse=True)
                    sees = torch.zeros(n + 20, dtype=torch.bool, device="cuda")
                    sees[at : (at + window if window else n)] = True
                    sees[n:] = False
                    assert torch.equal(lse[~sees], want_lse[~sees])
                    err = (o[~sees].float() - want[~sees].float()).abs()
                    # one key at a time adds its products in another order
                    within = err <= 2.0 ** -7 * want[~sees].float().abs() + 2.0 ** -16
                    assert within.all(), (D, window, bad, at, where)
                    if where == "v":
                        assert not torch.isfinite(o[sees][..., 5::7]).any()
                        assert torch.isfinite(o[sees][..., 4::7]).all()


def test_scores_of_minus_infinity(gpu_lib):
    """A row all of whose scores are -inf gives zeros and -inf."""
    q = torch.ones(3, 1, 64, dtype=torch.bfloat16, device="cuda")
    k = torch.ones(3, 1, 64, dtype=torch.bfloat16, device="cuda")
    k[0, 0, 0] = float("-inf")
    v = torch.full((3, 1, 64), 2.0, dtype=torch.bfloat16, device="cuda")
    o, lse = gpu_lib.prompt_attention(q, k, v, starts_of([3]), return_lse=True)
    assert (o[0] == 0).all() and torch.isneginf(lse[0]).all()
    assert (o[1:] == 2).all() and torch.isfinite(lse[1:]).all()


def test_growing_scores(gpu_lib):
    """Maxima that rise by more than the reference's slack again and again, and fall."""
    n, D = 700, 64
    r = gen("rising")
    q = ref.bf16(np.ones((n, 2, D)) + 0.1 * r.standard_normal((n, 2, D)))
    for ramp in (np.arange(n) / 20.0, -np.arange(n) / 20.0, np.where(np.arange(n) % 97 == 0, 40.0, -40.0)):
        k = ref.bf16(ramp[:, None, None] / 8 + 0.05 * r.standard_normal((n, 1, D)))
        v = ref.bf16(r.standard_normal((n, 1, D)))
        o, lse = gpu_lib.prompt_attention(q.cuda(), k.cuda(), v.cuda(), starts_of([n]), return_lse=True)
        check = Check(D ** -0.5, 0.0)
        check.sequence(o, lse, ref.f64(q), heads(k), heads(v), 0)
        check.done()


@pytest.mark.parametrize("lens,Hq,Hkv,D", [([77], 32, 8, 128), ([300, 5, 900], 4, 2, 64)])
def test_in_a_graph(gpu_lib, lens, Hq, Hkv, D):
    q, k, v = (t.cuda() for t in inputs(lens, Hq, Hkv, D))
    starts, o = starts_of(lens), torch.empty_like(q)
    lse = torch.empty(q.shape[:2], device="cuda")
    replay_equals_eager(lambda: gpu_lib.prompt_attention(q, k, v, starts, o=o, lse=lse), [o, lse])


def test_on_another_stream(gpu_lib):
    lens = [200, 31]
    q, k, v = (t.cuda() for t in inputs(lens, 8, 2, 128))
    want = gpu_lib.prompt_attention(q, k, v, starts_of(lens))
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got = [gpu_lib.prompt_attention(q, k, v, starts_of(lens)) for _ in range(3)]
    s.synchronize()
    assert all(torch.equal(g, want) for g in got)


def test_binding_refusals(gpu_lib):
    q = torch.zeros(4, 4, 64, dtype=torch.bfloat16, device="cuda")
    k = torch.zeros(4, 2, 64, dtype=torch.bfloat16, device="cuda")
    starts = torch.tensor([0, 4], dtype=torch.int32, device="cuda")
    f = gpu_lib.prompt_attention
    with pytest.raises(TypeError):
        f(q.float(), k, k, starts)
    with pytest.raises(ValueError, match="starts"):
        f(q, k, k, starts[:0])
    with pytest.raises(TypeError, match="starts"):
        f(q, k, k, starts.long())
    with pytest.raises(ValueError, match="k:"):
        f(q, k[:3], k[:3], starts)
    with pytest.raises(ValueError, match="v:"):
        f(q, k, k[:, :1], starts)
    with pytest.raises(ValueError, match="lie together"):
        f(q.transpose(1, 2).contiguous().transpose(1, 2), k, k, starts)
    wide = torch.zeros(4, 4, 68, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError, match="16 bytes"):
        f(wide[..., :64], k, k, starts)
    for bad in (dict(window=4, causal=False), dict(softcap=-1.0), dict(scale=float("nan")), dict(window=-1),
                dict(scale=1e38)):
        with pytest.raises(gpu_lib.Fp8LinError):
            f(q, k, k, starts, **bad)
    with pytest.raises(gpu_lib.Fp8LinError):
        f(q[:, :3], k, k, starts)  # three query heads on two key heads
    with pytest.raises(gpu_lib.Fp8LinError):
        f(q, k, k, starts, o=q)
    assert f(q[:0], k[:0], k[:0], starts * 0).shape == (0, 4, 64)
