"""kv_norm_rope_append and its e4m3 form against 64-bit references.

Tolerance (u = 2^-24): a head's squares are positive and added in chains of at most
16 fused steps and 4 sums, so their sum is within 20u; the mean, eps, root,
reciprocal and the two products make that at most 10u + 6u of a normed value.  A
rotated value adds 4u (|a| + |b|), so every value is within 20u of |a| + |b| (of
itself where nothing turns), before its one rounding.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

import layer_ref as ref
from test_graph_gpu import replay_equals_eager
from test_layer_gpu import U, assert_rounded, gen, holds, table

pytestmark = pytest.mark.gpu
MAX_POS = 300


def inputs(T, Hq, Hkv, D, rot, page, seed=0):
    r = gen(T, Hq, Hkv, D, rot, page, seed, "norm append")
    pages = -(-T // page) + 2
    qkv = ref.bf16(r.standard_normal((T, (Hq + 2 * Hkv) * D)) * 2.0 ** r.integers(-6, 7, (T, 1)))
    weights = [ref.bf16(1 + 0.3 * r.standard_normal(D)) for _ in range(2)]
    pos = r.integers(0, MAX_POS, T).astype(np.int32)
    slots = r.permutation(pages * page)[:T].astype(np.int64)
    if T > 3:
        slots[[1, T - 1]] = [-1, pages * page]  # neither is stored
    return qkv, weights, pos, slots, table(MAX_POS, rot), pages


def new_cache(pages, Hkv, page, D, fp8):
    dtype = torch.uint8 if fp8 else torch.bfloat16
    caches = [torch.full((pages, Hkv, page, D), 0x55 if fp8 else 7.0, dtype=dtype, device="cuda") for _ in range(2)]
    return caches + ([torch.full((pages, Hkv, page), -3.0, device="cuda") for _ in range(2)] if fp8 else [])


def expected(qkv, weights, pos, cs, Hq, Hkv, D, rot, interleaved, eps):
    """Normed and turned heads [T, Hq + Hkv, D] in 64 bits and the tolerance's unit."""
    x = ref.f64(qkv).reshape(len(pos), Hq + 2 * Hkv, D)[:, : Hq + Hkv].copy()
    for part, w in ((slice(0, Hq), weights[0]), (slice(Hq, Hq + Hkv), weights[1])):
        if w is not None:
            x[:, part] = ref.norm(x[:, part], None, ref.f64(w), eps)[1]
    c = cs.astype(np.float64)[pos]
    return ref.rotate(x, c[:, : rot // 2], c[:, rot // 2 :], rot, interleaved)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("normed", ["both", "queries", "keys", "none"])
@pytest.mark.parametrize("T,Hq,Hkv,D,rot,page,interleaved", [
    (1, 32, 8, 128, 128, 16, False), (1, 1, 1, 64, 64, 16, True), (2, 28, 4, 128, 64, 48, False),
    (57, 32, 8, 128, 128, 64, True), (130, 6, 2, 64, 32, 32, False), (33, 16, 1, 256, 256, 16, False),
    (19, 5, 5, 256, 128, 80, True), (40, 7, 7, 64, 16, 16, False), (11, 8, 2, 128, 0, 16, False),
    (9, 3, 1, 128, 112, 4096, True), (2051, 28, 4, 64, 32, 48, True), (1537, 16, 1, 256, 128, 32, False)])
def test_norm_append(gpu_lib, T, Hq, Hkv, D, rot, page, interleaved, normed, fp8):
    qkv, weights, pos, slots, cs, pages = inputs(T, Hq, Hkv, D, rot, page)
    weights = [w if normed in ("both", which) else None for w, which in zip(weights, ("queries", "keys"))]
    cache = new_cache(pages, Hkv, page, D, fp8)
    call = gpu_lib.kv_norm_rope_append_fp8 if fp8 else gpu_lib.kv_norm_rope_append
    dev = [qkv.cuda(), *(None if w is None else w.cuda() for w in weights), torch.from_numpy(pos).cuda(),
           torch.from_numpy(slots).cuda(), torch.from_numpy(cs).cuda()]
    q, keys = call(*dev, *cache, eps=1e-5, interleaved=interleaved, return_keys=True)
    other = [t.clone() for t in new_cache(pages, Hkv, page, D, fp8)]
    assert torch.equal(call(*dev, *other, eps=1e-5, interleaved=interleaved), q)  # the same without the keys' output
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(cache, other))
    turned, unit = expected(qkv, weights, pos, cs, Hq, Hkv, D, rot, interleaved, 1e-5)
    err = 20 * U * unit
    assert_rounded(q, turned[:, :Hq], err[:, :Hq], "q")
    assert_rounded(keys, turned[:, Hq:], err[:, Hq:], "keys")
    kept = (slots >= 0) & (slots < pages * page)
    at, off = slots[kept] // page, slots[kept] % page
    untouched = np.ones((pages, page), bool)
    untouched[at, off] = False
    values = ref.f64(qkv).reshape(T, -1, D)[:, Hq + Hkv :]
    for i, (rows, slack) in enumerate(((turned[:, Hq:], err[:, Hq:]), (values, np.zeros((T, Hkv, D))))):
        rows, slack, name = rows[kept], slack[kept], "kv"[i]
        host = cache[i].cpu()
        assert (host.permute(0, 2, 1, 3)[torch.from_numpy(untouched)] == (0x55 if fp8 else 7.0)).all()
        got = host[torch.from_numpy(at), :, torch.from_numpy(off)]
        if not fp8:
            assert_rounded(got, rows, slack, name)
            if name == "k":  # a cache line is the keys' output
                assert torch.equal(got, keys.cpu()[torch.from_numpy(kept)])
            continue
        s = cache[2 + i].cpu().numpy()
        assert (s.transpose(0, 2, 1)[untouched] == -3.0).all()
        s = s[at, :, off].astype(np.float64)
        amax = np.abs(rows).max(-1)
        holds(np.abs(s - amax / 448) <= slack.max(-1) / 448 + 2 * U * amax / 448, name + " scales")
        value = ref.e4m3_values(got) * s[..., None]
        step = np.maximum(2.0 ** -4 * np.abs(rows), 2.0 ** -10 * s[..., None]) * (1 + 2.0 ** -10)
        holds(np.abs(value - rows) <= step + 2 * slack + 2.0 ** -20 * np.abs(rows), name + " codes")


@pytest.mark.parametrize("fp8", [False, True])
def test_without_norms_it_is_the_plain_append(gpu_lib, fp8):
    T, Hq, Hkv, D, rot, page = 77, 12, 3, 128, 96, 48
    qkv, _, pos, slots, cs, pages = inputs(T, Hq, Hkv, D, rot, page)
    dev = [qkv.cuda(), torch.from_numpy(pos).cuda(), torch.from_numpy(slots).cuda(), torch.from_numpy(cs).cuda()]
    one, two = new_cache(pages, Hkv, page, D, fp8), new_cache(pages, Hkv, page, D, fp8)
    plain = gpu_lib.kv_rope_append_fp8 if fp8 else gpu_lib.kv_rope_append
    more = gpu_lib.kv_norm_rope_append_fp8 if fp8 else gpu_lib.kv_norm_rope_append
    assert torch.equal(plain(*dev, *one), more(dev[0], None, None, *dev[1:], *two, return_keys=True)[0])
    assert all(torch.equal(a, b) for a, b in zip(one, two))


def test_special_heads(gpu_lib):
    """A zero head stays zero by eps, an infinity gives NaN in its place and zeros beside it, a NaN its whole head; other
    heads and tokens are not touched.  Squares past fp32's range leave 0."""
    D, Hq, Hkv = 64, 2, 1
    x = torch.ones(5, 4, D)
    x[0, 0] = 0
    x[1, 0, 7] = float("inf")
    x[2, 2, 9] = float("nan")
    x[3, 1] = 2.0 ** 100
    w = torch.ones(D, dtype=torch.bfloat16, device="cuda")
    cs = torch.from_numpy(table(4, D)).cuda()
    cache = [torch.zeros(1, 1, 16, D, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    zero = torch.zeros(5, dtype=torch.int32, device="cuda")
    q, k = gpu_lib.kv_norm_rope_append(x.view(5, -1).bfloat16().cuda(), w, w, zero, torch.arange(5, device="cuda"), cs,
                                       *cache, eps=2.0 ** -10, return_keys=True)
    q, k = q.cpu().float(), k.cpu().float()
    assert (q[0, 0] == 0).all() and (q[3, 1] == 0).all()
    # at position 0 a pair turns to (a, b) itself, and its partner's product with the sine 0 is NaN
    assert torch.isnan(q[1, 0, [7, 39]]).all() and (q[1, 0, [i for i in range(D) if i not in (7, 39)]] == 0).all()
    assert torch.isnan(k[2, 0]).all()
    one = np.float64(1) / np.sqrt(1 + 2.0 ** -10)
    for t in (q[0, 1], q[1, 1], q[2], q[3, 0], q[4], k[[0, 1, 3, 4]]):
        assert (np.abs(t.numpy() - one) <= 2.0 ** -8).all()
    assert torch.equal(cache[0][0, 0, [0, 1, 3, 4]].cpu().float(), k[[0, 1, 3, 4], 0])


def test_in_a_graph(gpu_lib):
    T, Hq, Hkv, D, page = 33, 8, 2, 128, 16
    qkv, weights, pos, slots, cs, pages = inputs(T, Hq, Hkv, D, D, page)
    dev = [qkv.cuda(), *(w.cuda() for w in weights), torch.from_numpy(pos).cuda(), torch.from_numpy(slots).cuda(),
           torch.from_numpy(cs).cuda()]
    cache = new_cache(pages, Hkv, page, D, True)
    q = torch.empty(T, Hq, D, dtype=torch.bfloat16, device="cuda")
    k = torch.empty(T, Hkv, D, dtype=torch.bfloat16, device="cuda")
    # lines that no token has would not come back after the test clears the outputs
    kept = torch.from_numpy(slots[(slots >= 0) & (slots < pages * page)]).cuda()
    rows = [torch.empty(len(kept), Hkv, D, dtype=torch.uint8, device="cuda") for _ in range(2)]

    def step():
        gpu_lib.kv_norm_rope_append_fp8(*dev, *cache, return_keys=True, q=q, k=k)
        for i in range(2):
            rows[i].copy_(cache[i][kept // page, :, kept % page])

    replay_equals_eager(step, [q, k, *rows])


def test_binding_refusals(gpu_lib):
    qkv = torch.zeros(2, 4 * 64, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    pos, slots = torch.zeros(2, dtype=torch.int32, device="cuda"), torch.arange(2, device="cuda")
    cs = torch.zeros(4, 64, device="cuda")
    cache = [torch.zeros(1, 1, 16, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    for bad in (w[:32], w.float(), w.view(1, 64)):
        with pytest.raises((TypeError, ValueError), match="q_weight"):
            gpu_lib.kv_norm_rope_append(qkv, bad, w, pos, slots, cs, *cache)
        with pytest.raises((TypeError, ValueError), match="k_weight"):
            gpu_lib.kv_norm_rope_append(qkv, w, bad, pos, slots, cs, *cache)
    with pytest.raises(gpu_lib.Fp8LinError):
        gpu_lib.kv_norm_rope_append(qkv, w, w, pos, slots, cs, *cache, eps=-1.0)
    with pytest.raises(ValueError, match="k:"):
        gpu_lib.kv_norm_rope_append(qkv, w, w, pos, slots, cs, *cache, k=torch.empty_like(qkv))
