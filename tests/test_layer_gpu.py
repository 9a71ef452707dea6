"""The decoder-layer operators against plain 64-bit references (layer_ref.py).

Tolerances, from the number formats (u = 2^-24, half an fp32 ulp, relative):

* norm: the sum of squares adds at most 45 roundings in a chain, the root halves
  that, and the root, reciprocal and products add five more: v is within
  2^-18 |v|, its scale within 2^-18; a code adds half an e4m3 step (2^-4 of the
  value, or 2^-10 scales below the normal range);
* append: a rotated value is within 4u (|a| + |b|) of the exact one, plus its
  output rounding; value heads are exact;
* attention: with S the largest sum of scale |q_d k_d|, a score is within
  (D + 8) u S (plus the tanh's: 2^-20 softcap, and 2^-19 of a score); o is within twice that, plus
  2^-16 for the two-part weights and u for each token of a chain, times
  sum p |v|; lse within the score's error, 2^-19 and u for each token.

A bf16 output of a value known to within d lies between the bf16 roundings of
value - d and value + d: rounding is monotonic, so no output tolerance is added.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

import layer_ref as ref
from test_graph_gpu import replay_equals_eager

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def gen(*key):
    return np.random.default_rng([hash(k) % (1 << 31) if not isinstance(k, str) else sum(k.encode()) for k in key])


def holds(cond, what):
    cond = np.asarray(cond)
    if not cond.all():
        pytest.fail(f"{what}: {int((~cond).sum())} of {cond.size} values")


def assert_rounded(got, value, delta, what):
    """got (bf16) is a rounding of something within delta of value; 2^-23 covers the fp32 step of the casts here."""
    delta = delta + 2.0 ** -23 * np.abs(value)
    low, high = (torch.from_numpy(value + s * delta).to(torch.float32).bfloat16().double().numpy() for s in (-1, 1))
    got = ref.f64(got)
    holds((low <= got) & (got <= high), what)


# ------------------------------------------------------------------ norm

def norm_inputs(M, K, residual, seed=0):
    r = gen(M, K, residual, seed)
    channel = np.where(r.random(K) < 0.02, 20.0, 1.0)
    x = ref.bf16(r.standard_normal((M, K)) * channel)
    res = ref.bf16(3 * r.standard_normal((M, K)) * channel) if residual else None
    return x, res, ref.bf16(1 + 0.2 * r.standard_normal(K))


def check_codes(q, scale, v, slack=2.0 ** -17):
    """Codes with their scales (one for each run of v's last axis) against the 64-bit values v."""
    got = ref.e4m3_values(q).reshape(v.shape) * scale[..., None]
    bound = np.maximum(2.0 ** -4 * np.abs(v), 2.0 ** -10 * scale[..., None]) * (1 + 2.0 ** -10) + slack * np.abs(v)
    holds(np.abs(got - v) <= bound, "codes")


@pytest.mark.parametrize("scales", ["fp32", "ue8m0"])
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("M,K", [(1, 128), (5, 512), (3, 640), (9, 1024), (4, 1152), (2, 2048), (67, 2176), (1, 4096),
                                 (33, 7168), (3, 8192), (2, 8320), (3, 16384), (2, 18432), (1, 32768), (2, 40960)])
def test_norm(gpu_lib, M, K, residual, scales):
    x, res, w = norm_inputs(M, K, residual)
    call = gpu_lib.fp8_add_rmsnorm if scales == "fp32" else gpu_lib.fp8_add_rmsnorm_ue8m0
    h, y, q, s = call(x.cuda(), w.cuda(), None if res is None else res.cuda(), eps=1e-5, keep_y=True)
    torch.cuda.synchronize()
    _, v = ref.norm(ref.f64(x), None if res is None else ref.f64(res), ref.f64(w), 1e-5)
    if residual:
        assert torch.equal(h.cpu(), (x.float() + res.float()).bfloat16())
    else:
        assert h is None
    assert_rounded(y, v, 2.0 ** -18 * np.abs(v), "y")
    groups = v.reshape(M, K // 128, 128)
    amax = np.abs(groups).max(-1)
    if scales == "fp32":
        scale = ref.f64(s)
        holds(np.abs(scale - amax / 448) <= 2.0 ** -18 * amax / 448, "scales")
    else:
        scale = 2.0 ** (s.cpu().numpy().astype(np.float64) - 127)
        holds((448 * scale >= amax * (1 - 2.0 ** -18)) & (224 * scale < amax * (1 + 2.0 ** -18)), "scales")
    check_codes(q, scale, groups)


@pytest.mark.parametrize("K", [128, 1024, 4096, 8192, 65536])
def test_norm_codes_bit_exact(gpu_lib, K):
    """Rows whose root mean square is a power of two by the choice of eps, so that v = fl(h 2^-k w) is known in fp32
    and every code and scale can be held to the fp32 definition bit for bit."""
    M = 7
    r = gen(K, "exact")
    x = ref.bf16(r.integers(-2, 3, (M, K)))
    res = ref.bf16(r.integers(-1, 2, (M, K)))
    w = ref.bf16(r.standard_normal(K))
    h = x.float().numpy() + res.float().numpy()
    for m in range(M):
        mean = (h[m].astype(np.float64) ** 2).mean()
        eps = 16.0 - mean  # exact: a sum of small whole numbers over K, a power of two
        assert eps == np.float32(eps) and mean + np.float32(eps) == 16.0
        _, _, q, s = gpu_lib.fp8_add_rmsnorm(x[m : m + 1].cuda(), w.cuda(), res[m : m + 1].cuda(), eps=float(eps))
        v = (h[m] * np.float32(0.25) * w.float().numpy()).astype(np.float32).reshape(1, K // 128, 128)
        scale = (np.abs(v).max(-1) / np.float32(448)).astype(np.float32)
        assert np.array_equal(s.cpu().numpy(), scale)
        assert np.array_equal(q.cpu().numpy().reshape(v.shape), ref.e4m3_codes_f32(v, scale))
        e = gpu_lib.fp8_add_rmsnorm_ue8m0(x[m : m + 1].cuda(), w.cuda(), res[m : m + 1].cuda(), eps=float(eps))
        byte = e[3].cpu().numpy().astype(np.int64)
        pow2 = np.exp2(byte - 127.0)
        amax = np.abs(v).max(-1).astype(np.float64)
        assert (448 * pow2 >= amax).all() and ((448 * pow2 / 2 < amax) | (byte == 0)).all()
        assert np.array_equal(e[2].cpu().numpy().reshape(v.shape), ref.e4m3_codes_f32(v, pow2.astype(np.float32)))


def test_norm_in_place_and_without_codes(gpu_lib):
    x, res, w = norm_inputs(19, 4096, True)
    dx, dw, dres = x.cuda(), w.cuda(), res.cuda()
    h, y, q, s = gpu_lib.fp8_add_rmsnorm(dx, dw, dres, keep_y=True)
    stream = dres.clone()
    h2, y2, q2, s2 = gpu_lib.fp8_add_rmsnorm(dx, dw, stream, keep_y=True, h=stream)
    assert h2 is stream and torch.equal(stream, h) and torch.equal(y2, y) and torch.equal(q2, q) and torch.equal(s2, s)
    h3, y3, q3, s3 = gpu_lib.fp8_add_rmsnorm(dx, dw, dres, keep_y=True, quantize=False)
    assert q3 is None and s3 is None and torch.equal(y3, y) and torch.equal(h3, h)
    long = norm_inputs(3, 40960, True)
    lx, lres, lw = (t.cuda() for t in long)
    want = gpu_lib.fp8_add_rmsnorm(lx, lw, lres)
    got = gpu_lib.fp8_add_rmsnorm(lx, lw, lres, h=lres)
    for a, b in zip(want, got):
        assert (a is None and b is None) or torch.equal(a, b)


@pytest.mark.parametrize("M,K", [(8200, 7168), (16500, 3584)])
def test_norm_large(gpu_lib, M, K):
    """Inputs larger than the caches (read past them): sampled rows against the reference."""
    g = torch.Generator(device="cuda").manual_seed(3)
    x, res = (torch.randn(M, K, generator=g, device="cuda").bfloat16() for _ in range(2))
    w = ref.bf16(1 + 0.2 * gen(K, "large").standard_normal(K))
    h, y, q, s = gpu_lib.fp8_add_rmsnorm(x, w.cuda(), res, eps=1e-5, keep_y=True)
    rows = torch.cat([torch.arange(0, M, 97), torch.tensor([M - 1])])
    at = rows.cuda()
    xs, rs = x[at].cpu(), res[at].cpu()
    _, v = ref.norm(ref.f64(xs), ref.f64(rs), ref.f64(w), 1e-5)
    assert torch.equal(h[at].cpu(), (xs.float() + rs.float()).bfloat16())
    assert_rounded(y[at], v, 2.0 ** -18 * np.abs(v), "y")
    groups, scale = v.reshape(len(rows), K // 128, 128), ref.f64(s[at])
    holds(np.abs(scale - np.abs(groups).max(-1) / 448) <= 2.0 ** -18 * scale, "scales")
    check_codes(q[at], scale, groups)


@pytest.mark.parametrize("scales", ["fp32", "ue8m0"])
def test_norm_more_rows_than_one_launch(gpu_lib, scales):
    """More rows than one launch takes: repeated rows against a call of a few."""
    M, K, period = (1 << 21) + 777, 128, 4096
    x, res, w = (t.cuda() for t in norm_inputs(period, K, True, 5))
    call = gpu_lib.fp8_add_rmsnorm if scales == "fp32" else gpu_lib.fp8_add_rmsnorm_ue8m0
    want = call(x, w, res, keep_y=True)
    times = -(-M // period)
    got = call(x.repeat(times, 1)[:M], w, res.repeat(times, 1)[:M], keep_y=True)
    for a, b in zip(got, want):
        a, b = a.view(torch.uint8).view(M, -1), b.view(torch.uint8).view(period, -1)
        whole = M // period * period
        assert (a[:whole].view(-1, *b.shape) == b).all() and torch.equal(a[whole:], b[:M - whole])


def test_norm_special_rows(gpu_lib):
    """A zero row (eps keeps it zero), a row of tiny values, an infinity and a NaN: only their own rows are touched."""
    x = torch.ones(6, 512)
    x[1] = 0
    x[2] = 2.0 ** -120
    x[3, 200] = float("inf")
    x[4, 7] = float("nan")
    x = x.bfloat16()
    w = torch.ones(512, dtype=torch.bfloat16)
    h, y, q, s = gpu_lib.fp8_add_rmsnorm(x.cuda(), w.cuda(), eps=0.0 + 2.0 ** -100, keep_y=True)
    y, s, v = y.cpu().float(), s.cpu(), ref.e4m3_values(q)
    assert torch.equal(y[0], torch.ones(512)) and torch.equal(y[5], y[0])
    assert (y[1] == 0).all() and (s[1] == 0).all() and (v[1] == 0).all()
    small = 2.0 ** -120 / np.sqrt(2.0 ** -240 + 2.0 ** -100)
    assert np.allclose(y[2].numpy(), small, rtol=2.0 ** -8, atol=0) and np.allclose(
        v[2].reshape(4, 128) * s[2].numpy()[:, None], small, rtol=2.0 ** -4)
    # an infinite mean square: every finite value is 0, the infinite one NaN; a NaN spreads over its row
    assert torch.isnan(y[3, 200]) and (y[3, :200] == 0).all() and not torch.isfinite(s[3, 1])
    assert torch.isnan(y[4]).all() and torch.isnan(s[4]).all()
    e = gpu_lib.fp8_add_rmsnorm_ue8m0(x.cuda(), w.cuda(), eps=1e-5)[3].cpu()
    assert e[3, 1] == 255 and e[3, 0] == 0 and (e[4] == 255).all() and (e[0] == e[5]).all()


# ------------------------------------------------------------------ append

def table(max_pos, rot):
    angle = np.arange(max_pos)[:, None] * 10000.0 ** (-np.arange(0, rot, 2) / max(rot, 1))
    return np.concatenate([np.cos(angle), np.sin(angle)], -1).astype(np.float32)


def append_case(lib, T, Hq, Hkv, D, rot, page, fp8, interleaved, pages=None, seed=0):
    r = gen(T, Hq, Hkv, D, rot, page, seed)
    pages = pages or -(-T // page) + 2
    max_pos = 300
    qkv = ref.bf16(r.standard_normal((T, (Hq + 2 * Hkv) * D)))
    pos = r.integers(0, max_pos, T).astype(np.int32)
    slots = r.permutation(pages * page)[:T].astype(np.int64)
    if T > 3:
        slots[[1, T - 1]] = [-1, pages * page]  # neither is stored
    cs = table(max_pos, rot)
    dtype = torch.uint8 if fp8 else torch.bfloat16
    caches = [torch.full((pages, Hkv, page, D), 0x55 if fp8 else 7.0, dtype=dtype, device="cuda") for _ in range(2)]
    scales = [torch.full((pages, Hkv, page), -3.0, device="cuda") for _ in range(2)] if fp8 else []
    dev = [qkv.cuda(), torch.from_numpy(pos).cuda(), torch.from_numpy(slots).cuda(), torch.from_numpy(cs).cuda()]
    call = lib.kv_rope_append_fp8 if fp8 else lib.kv_rope_append
    q = call(*dev, *caches, *scales, interleaved=interleaved)
    torch.cuda.synchronize()
    x = ref.f64(qkv).reshape(T, Hq + 2 * Hkv, D)
    c = cs.astype(np.float64)[pos]
    turned, mag = ref.rotate(x[:, : Hq + Hkv], c[:, : rot // 2], c[:, rot // 2 :], rot, interleaved)
    err = 4 * U * mag
    assert_rounded(q, turned[:, :Hq], err[:, :Hq], "q")
    kept = (slots >= 0) & (slots < pages * page)
    at, off = slots[kept] // page, slots[kept] % page
    untouched = np.ones((pages, page), bool)
    untouched[at, off] = False
    want = {"k": (turned[:, Hq:], err[:, Hq:]), "v": (x[:, Hq + Hkv :], np.zeros((T, Hkv, D)))}
    for i, name in enumerate("kv"):
        rows, slack = want[name][0][kept], want[name][1][kept]
        got = caches[i].cpu()[torch.from_numpy(at), :, torch.from_numpy(off)]
        rest = caches[i].cpu().permute(0, 2, 1, 3)[torch.from_numpy(untouched)]
        assert (rest == (0x55 if fp8 else 7.0)).all()
        if not fp8:
            assert_rounded(got, rows, slack, name)
            if name == "v":
                assert np.array_equal(ref.f64(got), rows)
            continue
        s = scales[i].cpu().numpy()
        assert (s.transpose(0, 2, 1)[untouched] == -3.0).all()
        s = s[at, :, off]
        amax = np.abs(rows).max(-1)
        holds(np.abs(s - amax / 448) <= slack.max(-1) / 448 + 2 * U * amax / 448, name + " scales")
        codes = got.numpy()
        if name == "v":  # bf16 inputs: the fp32 definition holds bit for bit
            rows32 = rows.astype(np.float32)
            s32 = (np.abs(rows32).max(-1) / np.float32(448)).astype(np.float32)
            assert np.array_equal(s, s32) and np.array_equal(codes, ref.e4m3_codes_f32(rows32, s32))
        value = ref.e4m3_values(got) * s[..., None].astype(np.float64)
        step = np.maximum(2.0 ** -4 * np.abs(rows), 2.0 ** -10 * s[..., None]) * (1 + 2.0 ** -10)
        holds(np.abs(value - rows) <= step + 2 * slack + 2.0 ** -20 * np.abs(rows), name + " codes")


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("T,Hq,Hkv,D,rot,page,interleaved", [
    (1, 32, 8, 128, 128, 16, False), (1, 1, 1, 64, 64, 16, True), (2, 28, 4, 128, 64, 48, False),
    (57, 32, 8, 128, 128, 64, True), (130, 6, 2, 64, 32, 32, False), (33, 16, 1, 256, 256, 16, False),
    (19, 5, 5, 256, 128, 80, True), (40, 7, 7, 64, 16, 16, False), (11, 8, 2, 128, 0, 16, False),
    (9, 3, 1, 128, 112, 4096, True), (2051, 28, 4, 64, 32, 48, True), (4100, 6, 2, 128, 128, 16, False),
    (1537, 16, 1, 256, 128, 32, False), (515, 40, 8, 128, 128, 128, False), (3, 71, 71, 64, 48, 16, False)])
def test_append(gpu_lib, T, Hq, Hkv, D, rot, page, interleaved, fp8):
    append_case(gpu_lib, T, Hq, Hkv, D, rot, page, fp8, interleaved)


def test_append_positions_are_clamped(gpu_lib):
    """Positions past the table read its last row, negative ones its first."""
    cs = torch.from_numpy(table(10, 64)).cuda()
    qkv = ref.bf16(gen("clamp").standard_normal((4, 3 * 64))).cuda()
    qkv = qkv[:1].expand(4, -1).contiguous()
    cache = lambda: torch.zeros(1, 1, 16, 64, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    slots = torch.arange(4, device="cuda")
    q = gpu_lib.kv_rope_append(qkv, torch.tensor([-5, 0, 9, 1 << 30], dtype=torch.int32, device="cuda"), slots, cs,
                               cache(), cache())
    assert torch.equal(q[0], q[1]) and torch.equal(q[2], q[3]) and not torch.equal(q[0], q[2])


def test_append_special_values(gpu_lib):
    """Zero rows get scale 0 and zero codes; an infinity makes its row's scale infinite, a NaN NaN."""
    qkv = torch.ones(3, 3 * 64)
    qkv[0] = 0
    qkv[1, 64 + 5] = float("inf")
    qkv[2, 130] = float("nan")
    cs = torch.from_numpy(table(4, 64)).cuda()
    k, v = (torch.full((1, 1, 16, 64), 9, dtype=torch.uint8, device="cuda") for _ in range(2))
    ks, vs = (torch.full((1, 1, 16), 9.0, device="cuda") for _ in range(2))
    gpu_lib.kv_rope_append_fp8(qkv.bfloat16().cuda(), torch.zeros(3, dtype=torch.int32, device="cuda"),
                               torch.arange(3, device="cuda"), cs, k, v, ks, vs)
    ks, vs = ks.cpu().flatten(), vs.cpu().flatten()
    assert ks[0] == 0 and vs[0] == 0 and (ref.e4m3_values(k)[0, 0, 0] == 0).all()
    assert not torch.isfinite(ks[1]) and vs[1] == np.float32(1) / np.float32(448)
    assert torch.isnan(vs[2]) and torch.isfinite(ks[2]) and (ks[3:] == 9).all()


# ------------------------------------------------------------------ attention

def paged(r, lens, Hkv, D, page, fp8, window, spare=3, pages=None):
    """A cache whose live lines are random and everything else NaN, and its table (entries past the lengths out of
    range); returns device tensors and the live keys and values in 64 bits."""
    B = len(lens)
    per = [-(-n // page) for n in lens]
    total = pages or sum(per) + spare
    widest = max(1, max(per))
    order = r.permutation(total)[: sum(per)] if pages is None else total - 1 - np.arange(sum(per))
    dtype = torch.uint8 if fp8 else torch.bfloat16
    if pages is None:
        caches = [torch.full((total, Hkv, page, D), 0x7F if fp8 else float("nan"), dtype=dtype) for _ in range(2)]
        scales = [torch.full((total, Hkv, page), float("nan")) for _ in range(2)]
    else:
        caches = [torch.empty((total, Hkv, page, D), dtype=dtype, device="cuda") for _ in range(2)]
        scales = [torch.empty((total, Hkv, page), device="cuda") for _ in range(2)]
    table = np.where(r.random((B, widest)) < 0.5, -1, 1 << 30).astype(np.int32)
    live = []
    at = 0
    for b, n in enumerate(lens):
        ids = order[at : at + per[b]]
        at += per[b]
        table[b, : per[b]] = ids
        low = max(0, n - window) if window else 0
        kv = []
        for i in range(2):
            x = torch.from_numpy(r.standard_normal((n - low, Hkv, D)).astype(np.float32)).to(torch.bfloat16)
            t = np.arange(low, n)
            p, off = torch.from_numpy(ids[t // page].astype(np.int64)), torch.from_numpy(t % page)
            p, off = p.to(caches[i].device), off.to(caches[i].device)
            if fp8:
                s = (x.float().abs().amax(-1) / 448).numpy()
                codes = torch.from_numpy(ref.e4m3_codes_f32(x.float().numpy(), s))
                caches[i][p, :, off] = codes.to(caches[i].device)
                scales[i][p, :, off] = torch.from_numpy(s).to(caches[i].device)
                kv.append((ref.e4m3_values(codes) * s[..., None].astype(np.float64)).transpose(1, 0, 2))
            else:
                caches[i][p, :, off] = x.to(caches[i].device)
                kv.append(ref.f64(x).transpose(1, 0, 2))
        live.append(kv)
    dev = [c.cuda() for c in caches] + ([s.cuda() for s in scales] if fp8 else [])
    return dev, torch.from_numpy(table).cuda(), live


def attend_case(lib, lens, Hq, Hkv, D, page, fp8, window=0, softcap=0.0, max_len=None, sharp=1.5, pages=None, scale=None):
    r = gen(len(lens), sum(lens), Hq, Hkv, D, page, window)
    dev, table_, live = paged(r, lens, Hkv, D, page, fp8, window, pages=pages)
    if max_len is not None and table_.shape[1] * page < max_len:  # a wider table, its entries out of range
        more = -(-max_len // page) - table_.shape[1]
        table_ = torch.cat([table_, torch.full((len(lens), more), -9, dtype=torch.int32, device="cuda")], 1)
    q = ref.bf16(sharp * r.standard_normal((len(lens), Hq, D)))
    call = lib.paged_decode_attention_fp8 if fp8 else lib.paged_decode_attention
    args = (q.cuda(), *dev, table_, torch.tensor(lens, dtype=torch.int32, device="cuda"))
    kw = dict(window=window, softcap=softcap, max_len=max_len, scale=scale)
    print(f"attention lens={lens[:8]} Hq={Hq} Hkv={Hkv} D={D} page={page} fp8={fp8} {kw}", flush=True)
    o, lse = call(*args, **kw, return_lse=True)
    again = call(*args, **kw)
    torch.cuda.synchronize()
    assert torch.equal(o, again)  # deterministic, and the same without lse
    lse = ref.f64(lse)
    for b, n in enumerate(lens):
        want, want_lse, spread, size = ref.attention(ref.f64(q[b]), *live[b], D ** -0.5 if scale is None else scale,
                                                     softcap)
        score = (D + 8) * U * size + min(2.0 ** -20 * softcap, 2.0 ** -19 * size)
        assert_rounded(o[b], want, (2 * score + 2.0 ** -16 + n * U) * spread, f"o of row {b}, length {n}")
        if n == 0:
            assert (lse[b] == -np.inf).all()
        else:
            holds(np.abs(lse[b] - want_lse) <= score + 2.0 ** -19 + n * U + 2.0 ** -22 * np.abs(want_lse), "lse")


EDGES = [0, 1, 2, 15, 16, 17, 31, 32, 33, 47, 63, 64, 65, 100, 127, 128, 129, 255, 257, 511, 513]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("Hq,Hkv,D,page", [(32, 8, 128, 16), (28, 4, 64, 48), (16, 1, 256, 32), (3, 3, 128, 64),
                                           (40, 2, 128, 16), (33, 1, 64, 128), (64, 1, 128, 16), (70, 1, 256, 16),
                                           (8, 8, 64, 16), (10, 5, 256, 1024)])
def test_attention_edges(gpu_lib, Hq, Hkv, D, page, fp8):
    attend_case(gpu_lib, EDGES, Hq, Hkv, D, page, fp8)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("window,softcap", [(1, 0.0), (16, 0.0), (17, 30.0), (100, 0.0), (256, 5.0), (5000, 0.0),
                                            (0, 30.0), (1 << 40, 1.0)])
def test_attention_window_and_cap(gpu_lib, window, softcap, fp8):
    attend_case(gpu_lib, EDGES + [1500, 2047, 3001], 14, 2, 128, 48, fp8, window=window, softcap=softcap)


@pytest.mark.parametrize("softcap", [1e-40, 1e-3, 0.5, 300.0, 1e6, 1e30, 3e38])
def test_attention_caps_of_any_size(gpu_lib, softcap):
    """From caps that leave nothing of the scores to ones far above them, which change nothing."""
    attend_case(gpu_lib, [1, 40, 700], 6, 2, 64, 16, False, softcap=softcap)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("lens,Hq,Hkv,D,page", [([20001], 32, 8, 128, 16), ([9973, 3], 8, 1, 64, 64),
                                                ([5000, 0, 4999, 1], 16, 16, 64, 48), ([8193] * 3, 4, 2, 256, 16),
                                                ([4097], 1, 1, 128, 4096)])
def test_attention_long(gpu_lib, lens, Hq, Hkv, D, page, fp8):
    attend_case(gpu_lib, lens, Hq, Hkv, D, page, fp8)


def ragged(kind):
    r = gen("ragged", kind)
    if kind == "few long among short":
        return [int(x) for x in np.where(r.random(150) < 0.05, r.integers(500, 3000, 150), r.integers(0, 90, 150))]
    if kind == "all one":
        return [1] * 70
    if kind == "one long":
        return [40, 9000]
    if kind == "fewer tiles than waves":
        return [3, 0, 64]
    return [int(x) for x in 2 ** r.uniform(0, 11, 67)]  # spread over the logarithm


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("Hq,Hkv,D,page,window", [(32, 8, 128, 16, 0), (20, 1, 128, 48, 0), (6, 3, 64, 16, 1500),
                                                  (36, 2, 64, 16, 0), (8, 2, 256, 32, 0)])
@pytest.mark.parametrize("kind", ["few long among short", "all one", "one long", "fewer tiles than waves", "spread"])
def test_attention_ragged(gpu_lib, kind, Hq, Hkv, D, page, window, fp8):
    """Batches whose work is divided over the workgroups in even shares (host bounds above the lengths): shares
    with many rows, rows with many shares, and shares without work."""
    lens = ragged(kind)
    for bound in (max(4096, max(lens)), 1 << 17):  # by the grid for small batches, in even shares
        attend_case(gpu_lib, lens, Hq, Hkv, D, page, fp8, window=window, max_len=bound)


def test_attention_batch(gpu_lib):
    attend_case(gpu_lib, [(37 * i) % 400 for i in range(300)], 8, 2, 64, 16, True)


@pytest.mark.parametrize("scale,sharp", [(1.0, 6.0), (-0.3, 2.0), (0.0, 1.0)])
def test_attention_scales(gpu_lib, scale, sharp):
    """Sharp scores (weights that underflow beside the largest), a negative scale, and none."""
    attend_case(gpu_lib, [5, 300, 1025], 8, 2, 128, 16, False, scale=scale, sharp=sharp)


def test_attention_max_len(gpu_lib):
    """A bound below the table's width gives the same result; longer sequences are cut to it."""
    lens = [100, 700, 513]
    r = gen("max_len")
    dev, table_, _ = paged(r, lens, 2, 128, 16, False, 0)
    q = ref.bf16(r.standard_normal((3, 8, 128))).cuda()
    seq = torch.tensor(lens, dtype=torch.int32, device="cuda")
    full = gpu_lib.paged_decode_attention(q, *dev, table_, seq, max_len=700)
    wide = torch.cat([table_, torch.full((3, 5000), -7, dtype=torch.int32, device="cuda")], 1).contiguous()
    free = gpu_lib.paged_decode_attention(q, *dev, wide, seq)
    assert (full.float() - free.float()).abs().max() <= 2.0 ** -8 * full.float().abs().max()
    cut = gpu_lib.paged_decode_attention(q, *dev, table_, seq, max_len=513)
    again = gpu_lib.paged_decode_attention(q, *dev, table_, seq.clamp(max=513), max_len=513)
    assert torch.equal(cut, again)
    none = gpu_lib.paged_decode_attention(q, *dev, table_, torch.full_like(seq, -3), max_len=0)
    assert (none == 0).all()


def test_attention_infinite_scores(gpu_lib):
    """Keys of minus infinity give weight 0 (a mask written into the keys); where every key is so nothing is left and
    the row is 0; a NaN key makes its row NaN.  Other rows are untouched."""
    D, page, n = 64, 16, 40
    k = torch.zeros(12, 1, page, D, dtype=torch.bfloat16)
    v = torch.ones(12, 1, page, D, dtype=torch.bfloat16)
    v[0] = 3
    k[0, 0, :, 0] = float("-inf")      # the first page of row 0
    k[3:6, 0, :, 0] = float("-inf")    # all of row 1
    k[6, 0, 3, 1] = float("nan")
    table_ = torch.arange(12, dtype=torch.int32).view(4, 3).cuda()
    q = torch.ones(4, 2, D, dtype=torch.bfloat16).cuda()
    o = gpu_lib.paged_decode_attention(q, k.cuda(), v.cuda(), table_, torch.full((4,), n, dtype=torch.int32).cuda())
    o = o.cpu().float()
    assert (o[0] == 1).all() and torch.isnan(o[2]).all() and (o[3] == 1).all()
    assert (o[1] == 0).all()


def test_attention_more_rows_than_a_grid(gpu_lib):
    """More than 2^24 rows (a sequence's key heads), all of one token or none: the token's value, or zeros."""
    B, H, D, page = 65535, 257, 64, 16
    g = torch.Generator(device="cuda").manual_seed(11)
    k, v = (torch.randn(3, H, page, D, generator=g, device="cuda").bfloat16() for _ in range(2))
    q = torch.randn(H, D, generator=g, device="cuda").bfloat16().expand(B, H, D).contiguous()
    pages = (torch.arange(B, dtype=torch.int32, device="cuda") % 3).view(B, 1).contiguous()
    lens = (torch.arange(B, dtype=torch.int32, device="cuda") % 5 != 0).int()
    o = gpu_lib.paged_decode_attention(q, k, v, pages, lens)
    want = v[:, :, 0]
    for b0 in range(0, B, 8192):  # in pieces, for memory
        b1 = min(B, b0 + 8192)
        piece = want[pages[b0:b1, 0].long()] * lens[b0:b1].view(-1, 1, 1)
        assert (o[b0:b1] == piece).all()


@pytest.mark.parametrize("fp8", [False, True])
def test_attention_and_append_past_32_bits(gpu_lib, fp8):
    """A cache of more than 2^32 elements, its last pages in use."""
    pages = 270000 if not fp8 else 530000  # 4.4e9 and 8.7e9 elements of 16 x 8 x 128
    attend_case(gpu_lib, [50, 33], 16, 8, 128, 16, fp8, pages=pages)
    torch.cuda.empty_cache()
    kind = torch.uint8 if fp8 else torch.bfloat16
    k, v = (torch.empty(pages, 8, 16, 128, dtype=kind, device="cuda") for _ in range(2))
    sc = [torch.empty(pages, 8, 16, device="cuda") for _ in range(2)] if fp8 else []
    qkv = ref.bf16(gen("far").standard_normal((2, 32 * 128))).cuda()
    slots = torch.tensor([pages * 16 - 1, 5], device="cuda")
    cs = torch.from_numpy(table(4, 128)).cuda()
    pos = torch.zeros(2, dtype=torch.int32, device="cuda")
    (gpu_lib.kv_rope_append_fp8 if fp8 else gpu_lib.kv_rope_append)(qkv, pos, slots, cs, k, v, *sc)
    rows = qkv.view(2, 32, 128)
    for got, want in ((v[-1, :, 15], rows[0, 24:]), (v[0, :, 5], rows[1, 24:]), (k[-1, :, 15], rows[0, 16:24])):
        if fp8:
            s = want.float().abs().amax(-1, keepdim=True) / 448
            got = got.contiguous().view(torch.float8_e4m3fn).float() * s
            assert ((got - want.float()).abs() <= 2.0 ** -4 * want.float().abs() + 2.0 ** -9 * s).all()
        else:
            assert torch.equal(got, want)
    del k, v, sc
    torch.cuda.empty_cache()


# ------------------------------------------------------------------ streams and graphs

def test_layer_graph_replay(gpu_lib):
    x, res, w = norm_inputs(33, 4096, True)
    x, res, w = x.cuda(), res.cuda(), w.cuda()
    h, q = torch.empty_like(x), torch.empty(33, 4096, dtype=torch.uint8, device="cuda")
    s = torch.empty(33, 32, device="cuda")
    replay_equals_eager(lambda: gpu_lib.fp8_add_rmsnorm(x, w, res, h=h, q=q, s=s), [h, q, s])
    for lens, Hkv in (([6000, 17, 0, 3000], 2), ([(61 * i) % 3000 for i in range(48)], 8)):  # by the grid, in shares
        r = gen("graph", Hkv)
        dev, table_, _ = paged(r, lens, Hkv, 128, 16, True, 0)
        qq = ref.bf16(r.standard_normal((len(lens), 4 * Hkv, 128))).cuda()
        seq = torch.tensor(lens, dtype=torch.int32, device="cuda")
        o, lse = torch.empty_like(qq), torch.empty(len(lens), 4 * Hkv, device="cuda")
        replay_equals_eager(lambda: gpu_lib.paged_decode_attention_fp8(qq, *dev, table_, seq, return_lse=True, o=o,
                                                                       lse=lse), [o, lse])


def test_layer_on_side_streams(gpu_lib):
    """Two streams at once, inputs made on another stream, each call's scratch its own."""
    r = gen("streams")
    dev, table_, _ = paged(r, [7000], 2, 128, 16, False, 0)
    seq = torch.tensor([7000], dtype=torch.int32, device="cuda")
    qs = [ref.bf16(r.standard_normal((1, 16, 128))).cuda() for _ in range(2)]
    want = [gpu_lib.paged_decode_attention(q, *dev, table_, seq) for q in qs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for _ in range(8):
        for q, st in zip(qs, streams):
            st.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(st):
                got.append(gpu_lib.paged_decode_attention(q, *dev, table_, seq))
    torch.cuda.synchronize()
    for i, g in enumerate(got):
        assert torch.equal(g, want[i % 2])
