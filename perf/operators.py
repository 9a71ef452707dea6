"""Measured cases of the decoder-layer operators that sit between the FP8 linears.

Three operators, each with its plain form (elementary torch operations in 32 bits, rounded once at the end) and with
the library's call:

* ``norm``: residual addition, root-mean-square norm and e4m3 quantization in 1x128 groups, the input of an FP8 linear;
* ``append``: rotary position embedding of the query and key heads of a QKV projection, and the append of keys and
  values to a paged cache (bf16, or e4m3 with one scale for each token and head);
* ``attend``: attention of one new token of each sequence over the paged cache.

``own`` chooses the side.  A case is a dict of plain values; ``prepare`` makes its inputs on the GPU from a seed, ``run``
is one pass, ``exact`` the same outputs from the definitions in 64 bits.  Outputs held in 8 bits are returned as
float8 tensors, beside their scales.
"""
from __future__ import annotations

import math

import numpy as np
import torch

own = False

E4M3_MAX = 448.0
GROUP = 128
MAX_POSITION = 16384  # rows of the rotation table
DEVICE = "cuda"


def listed():
    return [
        # one decoded token through the norm before a 4096-wide projection: latency
        dict(name="norm_token", op="norm", rows=1, width=4096, residual=True, scales="fp32", keep=False),
        # a decode batch of odd size, 7168 wide, power-of-two scales
        dict(name="norm_batch", op="norm", rows=57, width=7168, residual=True, scales="ue8m0", keep=False),
        # an odd-sized prompt's first norm: no residual yet, the bf16 output kept for a layer that is not quantized
        dict(name="norm_prompt", op="norm", rows=4093, width=4096, residual=False, scales="fp32", keep=True),
        # a large prefill batch inside the network, 7168 wide
        dict(name="norm_prefill", op="norm", rows=8192, width=7168, residual=True, scales="fp32", keep=False),
        # one decoded token: latency of the rotation and append
        dict(name="append_token", op="append", tokens=1, padded=0, prompts=1, q_heads=32, kv_heads=8, head_dim=128,
             rotated=128, interleaved=False, page=16, cache="bf16"),
        # a decode batch padded to 64 rows, into an e4m3 cache
        dict(name="append_batch", op="append", tokens=64, padded=7, prompts=57, q_heads=32, kv_heads=8, head_dim=128,
             rotated=128, interleaved=False, page=64, cache="e4m3"),
        # three packed prompts of odd lengths, neighbouring pairs rotated in half of each 64-wide head
        dict(name="append_prompts", op="append", tokens=4093, padded=0, prompts=3, q_heads=28, kv_heads=4,
             head_dim=64, rotated=32, interleaved=True, page=48, cache="bf16"),
        # a long prefill into an e4m3 cache
        dict(name="append_prefill", op="append", tokens=8192, padded=0, prompts=4, q_heads=32, kv_heads=8,
             head_dim=128, rotated=128, interleaved=False, page=16, cache="e4m3"),
        # one chat user, a short cache: latency
        dict(name="attend_token", op="attend", batch=1, empty=0, shortest=777, longest=777, q_heads=32, kv_heads=8,
             head_dim=128, page=16, cache="bf16", window=0, softcap=0.0),
        # one user, a very long cache: the split over the cache's length
        dict(name="attend_long", op="attend", batch=1, empty=0, shortest=131072, longest=131072, q_heads=32,
             kv_heads=8, head_dim=128, page=16, cache="bf16", window=0, softcap=0.0),
        # a serving batch of ragged lengths over an e4m3 cache
        dict(name="attend_batch", op="attend", batch=64, empty=0, shortest=1, longest=8192, q_heads=32, kv_heads=8,
             head_dim=128, page=64, cache="e4m3", window=0, softcap=0.0),
        # heads of their own keys, 64 wide, a sliding window and capped scores, two rows of the batch unused
        dict(name="attend_window", op="attend", batch=37, empty=2, shortest=5, longest=6000, q_heads=16, kv_heads=16,
             head_dim=64, page=48, cache="bf16", window=1024, softcap=30.0),
    ]


def _spread(rng, low, high):
    """A whole number of [low, high], spread over its logarithm."""
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


HEADS = [(32, 8), (28, 4), (16, 16), (16, 1), (40, 8), (64, 8), (6, 2), (10, 10), (32, 1)]
PAGES = [16, 32, 48, 64, 128]


def draw(rng):
    op = rng.choice(["norm", "append", "attend"])
    if op == "norm":
        width = GROUP * rng.choice([n for n in (_spread(rng, 1, 128), 56) if n != 24])
        rows = _spread(rng, 1, max(1, min(16384, 8192 * 7168 // width)))
        return dict(op=op, rows=rows, width=width, residual=rng.random() < 0.7, scales=rng.choice(["fp32", "ue8m0"]),
                    keep=rng.random() < 0.3)
    q_heads, kv_heads = rng.choice(HEADS)
    head_dim = rng.choice([64, 128, 128, 256] if q_heads + 2 * kv_heads != 48 else [128, 256])
    page, cache = rng.choice(PAGES), rng.choice(["bf16", "e4m3"])
    if op == "append":
        most = 8192 * 48 * 128 // ((q_heads + 2 * kv_heads) * head_dim)
        tokens = _spread(rng, 1, most)
        prompts = tokens if rng.random() < 0.4 and tokens <= 256 else min(tokens, rng.randint(1, 5))
        padded = rng.randint(0, (tokens - prompts) // 8) if tokens > prompts else 0
        return dict(op=op, tokens=tokens, padded=padded, prompts=prompts, q_heads=q_heads, kv_heads=kv_heads,
                    head_dim=head_dim, rotated=rng.choice([head_dim, head_dim, head_dim // 2]),
                    interleaved=rng.random() < 0.4, page=page, cache=cache)
    batch = _spread(rng, 1, 256)
    most = 64 * 8192 * 8 * 128 // (batch * kv_heads * head_dim)
    most = min(most, 64 * 8192 * 32 * 128 // (batch * q_heads * head_dim), 131072)
    longest = _spread(rng, 1, max(1, most))
    return dict(op=op, batch=batch, empty=rng.randint(0, batch // 8), shortest=max(1, int(longest * rng.random())),
                longest=longest, q_heads=q_heads, kv_heads=kv_heads, head_dim=head_dim, page=page, cache=cache,
                window=rng.choice([0, 0, _spread(rng, 1, 4096)]), softcap=rng.choice([0.0, 0.0, 30.0]))


def _lengths(case):
    """The sequences' lengths, in order: a few unused rows, then lengths that crowd near the shortest."""
    n, e = case["batch"], case["empty"]
    u = np.linspace(0.0, 1.0, n - e) if n - e > 1 else np.ones(n - e)
    full = case["shortest"] + np.rint((case["longest"] - case["shortest"]) * u * u).astype(np.int64)
    return np.concatenate([np.zeros(e, np.int64), full])


def work(case):
    if case["op"] == "norm":
        m, k = case["rows"], case["width"]
        scale = 4 if case["scales"] == "fp32" else 1
        per = 2 + 1 + scale / GROUP + (4 if case["residual"] else 0) + (2 if case["keep"] else 0)
        return {"bytes": m * k * per + 2 * k, "flops": m * k * 6}
    hq, hkv, d = case["q_heads"], case["kv_heads"], case["head_dim"]
    size = 2 if case["cache"] == "bf16" else 1 + 4 / d
    if case["op"] == "append":
        t, stored = case["tokens"], case["tokens"] - case["padded"]
        moved = t * (hq + 2 * hkv) * d * 2 + t * hq * d * 2 + stored * 2 * hkv * d * size + t * 12
        return {"bytes": moved + min(t, MAX_POSITION) * case["rotated"] * 4, "flops": t * (hq + hkv) * d * 6}
    lens = _lengths(case)
    seen = int(np.minimum(lens, case["window"]).sum() if case["window"] else lens.sum())
    b = case["batch"]
    table = int(np.ceil(lens / case["page"]).sum()) * 4
    return {"bytes": seen * hkv * d * 2 * size + b * hq * (d * 4 + 4) + table + 4 * b, "flops": seen * hq * d * 4}


def _generator(seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(int(seed) * 7919 + 17)
    return g


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device=DEVICE, dtype=torch.float32)


def _to_cache(x):
    """Rows of heads as an e4m3 cache holds them: codes, and one scale for each row."""
    s = x.float().abs().amax(-1) / E4M3_MAX
    return (x.float() / torch.where(s == 0, 1.0, s)[..., None]).to(torch.float8_e4m3fn).view(torch.uint8), s


def prepare(case, seed):
    g = _generator(seed)
    st = dict(case)
    if case["op"] == "norm":
        m, k = case["rows"], case["width"]
        # activations with a few channels of large values, as decoder layers have them
        channel = torch.where(torch.rand(k, generator=g, device=DEVICE) < 0.01, 20.0, 1.0)
        st["x"] = (_normal(g, m, k) * channel).bfloat16()
        st["res"] = (3.0 * _normal(g, m, k) * channel).bfloat16() if case["residual"] else None
        st["weight"] = (1.0 + 0.2 * _normal(g, k)).bfloat16()
        st["eps"] = 1e-5
        return st
    hq, hkv, d, page = case["q_heads"], case["kv_heads"], case["head_dim"], case["page"]
    if case["op"] == "append":
        t, r = case["tokens"], case["rotated"]
        real, n = t - case["padded"], case["prompts"]
        sizes = torch.full((n,), real // n, dtype=torch.int64)
        sizes[: real % n] += 1
        sizes = sizes.to(DEVICE)
        start = (torch.rand(n, generator=g, device=DEVICE) * (MAX_POSITION - sizes)).long()
        prompt = torch.repeat_interleave(torch.arange(n, device=DEVICE), sizes, output_size=real)
        inside = torch.arange(real, device=DEVICE) - (torch.cumsum(sizes, 0) - sizes)[prompt]
        position = start[prompt] + inside
        pages = real // page + 2 * n + 1
        order = torch.randperm(pages, generator=g, device=DEVICE)
        held = sizes // page + 2  # pages of each prompt, at most
        local = position // page - (start // page)[prompt]
        slot = order[(torch.cumsum(held, 0) - held)[prompt] + local] * page + position % page
        st["qkv"] = _normal(g, t, (hq + 2 * hkv) * d).bfloat16()
        st["positions"] = torch.zeros(t, dtype=torch.int32, device=DEVICE)
        st["positions"][:real] = position.int()
        st["slots"] = torch.full((t,), -1, dtype=torch.int64, device=DEVICE)  # rows of padding are not stored
        st["slots"][:real] = slot
        angle = torch.arange(MAX_POSITION, device=DEVICE, dtype=torch.float64)[:, None] \
            * 10000.0 ** (-torch.arange(0, r, 2, device=DEVICE, dtype=torch.float64) / r)
        st["cos_sin"] = torch.cat([angle.cos(), angle.sin()], -1).float()
        kind = torch.bfloat16 if case["cache"] == "bf16" else torch.uint8
        for name in ("k", "v"):
            st[name + "_cache"] = torch.zeros(pages, hkv, page, d, dtype=kind, device=DEVICE)
            if case["cache"] == "e4m3":
                st[name + "_scale"] = torch.zeros(pages, hkv, page, dtype=torch.float32, device=DEVICE)
        return st
    lens = _lengths(case)
    lens = torch.from_numpy(lens).to(DEVICE)[torch.randperm(case["batch"], generator=g, device=DEVICE)]
    per = (lens + page - 1) // page
    widest = max(1, -(-case["longest"] // page))
    total = int(np.ceil(_lengths(case) / page).sum()) + 3
    order = torch.randperm(total, generator=g, device=DEVICE)
    at = (torch.cumsum(per, 0) - per)[:, None] + torch.arange(widest, device=DEVICE)
    used = torch.arange(widest, device=DEVICE) < per[:, None]
    st["block_table"] = torch.where(used, order[torch.where(used, at, 0)], 0).int()
    st["seq_lens"] = lens.int()
    st["q"] = (1.5 * _normal(g, case["batch"], hq, d)).bfloat16()
    for name in ("k", "v"):
        x = torch.randn(total, hkv, page, d, generator=g, device=DEVICE, dtype=torch.bfloat16)
        if case["cache"] == "bf16":
            st[name + "_cache"] = x
        else:
            st[name + "_cache"], st[name + "_scale"] = _to_cache(x)
        del x
    return st


def run(st):
    return {"norm": _norm, "append": _append, "attend": _attend}[st["op"]](st)


def _norm(st):
    pow2 = st["scales"] == "ue8m0"
    if own:
        import sparse_gemm_linears_amd as sgl
        call = sgl.fp8_add_rmsnorm_ue8m0 if pow2 else sgl.fp8_add_rmsnorm
        h, y, q, s = call(st["x"], st["weight"], st["res"], eps=st["eps"], keep_y=st["keep"])
    else:
        m, k = st["x"].shape
        x = st["x"].float()
        if st["res"] is not None:
            x = x + st["res"].float()
        v = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + st["eps"]) * st["weight"].float()
        v3 = v.view(m, k // GROUP, GROUP)
        amax = v3.abs().amax(-1)
        if pow2:
            bits = amax.view(torch.int32)
            e = ((bits >> 23) - 8 + ((bits & 0x7FFFFF) > 0x600000).int()).clamp(min=0)
            s, div = e.to(torch.uint8), torch.exp2((e - 127).float())
        else:
            s = amax / E4M3_MAX
            div = torch.where(s == 0, 1.0, s)
        q = (v3 / div[..., None]).to(torch.float8_e4m3fn).view(m, k)
        h = x.bfloat16() if st["res"] is not None else None
        y = v.bfloat16() if st["keep"] else None
    s = s.view(torch.float8_e8m0fnu) if pow2 else s
    return {"h": h, "y": y, "codes": q.view(torch.float8_e4m3fn), "scales": s}


def _rotate(x, cos, sin, r, interleaved):
    """The rotation of the first r values of each head: pairs (i, i + r/2), or neighbours where interleaved."""
    if interleaved:
        a, b = x[..., 0:r:2], x[..., 1:r:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = x[..., : r // 2], x[..., r // 2 : r]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([turned, x[..., r:]], -1)


def _append(st):
    hq, hkv, r = st["q_heads"], st["kv_heads"], st["rotated"]
    narrow = st["cache"] == "e4m3"
    if own:
        import sparse_gemm_linears_amd as sgl
        if narrow:
            q = sgl.kv_rope_append_fp8(st["qkv"], st["positions"], st["slots"], st["cos_sin"], st["k_cache"],
                                       st["v_cache"], st["k_scale"], st["v_scale"], interleaved=st["interleaved"])
        else:
            q = sgl.kv_rope_append(st["qkv"], st["positions"], st["slots"], st["cos_sin"], st["k_cache"],
                                   st["v_cache"], interleaved=st["interleaved"])
    else:
        t, page, real = st["tokens"], st["page"], st["tokens"] - st["padded"]
        x = st["qkv"].float().view(t, hq + 2 * hkv, -1)
        table = st["cos_sin"][st["positions"].long()][:, None]
        turned = _rotate(x[:, : hq + hkv], table[..., : r // 2], table[..., r // 2 :], r, st["interleaved"])
        q = turned[:, :hq].bfloat16()
        at, off = st["slots"][:real] // page, st["slots"][:real] % page
        for name, rows in (("k", turned[:real, hq:]), ("v", x[:real, hq + hkv :])):
            if narrow:
                codes, s = _to_cache(rows)
                st[name + "_cache"][at, :, off] = codes
                st[name + "_scale"][at, :, off] = s
            else:
                st[name + "_cache"][at, :, off] = rows.bfloat16()
    if not narrow:
        return {"q": q, "k": st["k_cache"], "v": st["v_cache"]}
    return {"q": q, "k": st["k_cache"].view(torch.float8_e4m3fn), "v": st["v_cache"].view(torch.float8_e4m3fn),
            "k_scale": st["k_scale"], "v_scale": st["v_scale"]}


def _attend(st):
    d, narrow = st["head_dim"], st["cache"] == "e4m3"
    if own:
        import sparse_gemm_linears_amd as sgl
        more = dict(softcap=st["softcap"], window=st["window"], max_len=st["longest"], return_lse=True)
        if narrow:
            o, lse = sgl.paged_decode_attention_fp8(st["q"], st["k_cache"], st["v_cache"], st["k_scale"],
                                                    st["v_scale"], st["block_table"], st["seq_lens"], **more)
        else:
            o, lse = sgl.paged_decode_attention(st["q"], st["k_cache"], st["v_cache"], st["block_table"],
                                                st["seq_lens"], **more)
        return {"o": o, "lse": lse}
    b, hq = st["q"].shape[:2]
    hkv, table = st["kv_heads"], st["block_table"].long()

    def rows(name):
        x = st[name + "_cache"][table]  # [batch, pages, kv heads, page, d]
        x = x.view(torch.float8_e4m3fn).float() * st[name + "_scale"][table][..., None] if narrow else x.float()
        return x.transpose(1, 2).reshape(b, hkv, -1, d)

    k, v = rows("k"), rows("v")
    at, lens = torch.arange(k.shape[2], device=DEVICE), st["seq_lens"].long()[:, None]
    live = at < lens
    if st["window"]:
        live = live & (at >= lens - st["window"])
    score = torch.matmul(st["q"].float().view(b, hkv, hq // hkv, d), k.transpose(-1, -2)) / math.sqrt(d)
    if st["softcap"]:
        score = st["softcap"] * torch.tanh(score / st["softcap"])
    score = score.masked_fill(~live[:, None, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - torch.where(torch.isfinite(top), top, 0.0))
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v) / torch.where(total == 0, 1.0, total)
    lse = torch.where(total == 0, -math.inf, top + torch.log(total))
    return {"o": o.view(b, hq, d).bfloat16(), "lse": lse.view(b, hq)}


def exact(case, seed):
    """The outputs in 64 bits.  Codes are given as the quotients that they round, so an error is the rounding's own."""
    st = prepare(case, seed)
    f = torch.float64
    if case["op"] == "norm":
        m, k = st["x"].shape
        h = st["x"].to(f) + (st["res"].to(f) if case["residual"] else 0.0)
        y = h / torch.sqrt(torch.linalg.vecdot(h, h)[:, None] / k + st["eps"]) * st["weight"].to(f)
        groups = y.unflatten(1, (-1, GROUP))
        amax = torch.linalg.vector_norm(groups, math.inf, dim=-1)
        if case["scales"] == "ue8m0":
            mantissa, power = torch.frexp(amax)  # 448 = 0.875 * 2^9
            s = torch.ldexp(torch.ones_like(amax), (power - 9 + (mantissa > 0.875).int()).clamp(min=-127))
        else:
            s = amax / E4M3_MAX
        codes = (groups / torch.where(s == 0, 1.0, s)[..., None]).flatten(1)
        return {"h": h if case["residual"] else None, "y": y if case["keep"] else None, "codes": codes, "scales": s}
    hq, hkv, d, page = case["q_heads"], case["kv_heads"], case["head_dim"], case["page"]
    if case["op"] == "append":
        t, r, real = case["tokens"], case["rotated"], case["tokens"] - case["padded"]
        half = r // 2
        first = torch.arange(half, device=DEVICE) * (2 if case["interleaved"] else 1)
        second = first + (1 if case["interleaved"] else half)
        x = st["qkv"].to(f).view(t, hq + 2 * hkv, d)
        cs = st["cos_sin"].to(f)[st["positions"].long()]
        z = torch.complex(x[..., first], x[..., second])[:, : hq + hkv] * torch.complex(cs[:, :half], cs[:, half:])[:, None]
        x[:, : hq + hkv, first], x[:, : hq + hkv, second] = z.real, z.imag
        out = {"q": x[:, :hq]}
        for name, rows in (("k", x[:real, hq : hq + hkv]), ("v", x[:real, hq + hkv :])):
            cache = torch.zeros(st[name + "_cache"].shape, dtype=f, device=DEVICE).transpose(1, 2).flatten(0, 1)
            if case["cache"] == "e4m3":
                s = rows.abs().amax(-1) / E4M3_MAX
                scale = torch.zeros(cache.shape[:2], dtype=f, device=DEVICE)
                scale[st["slots"][:real]] = s
                out[name + "_scale"] = scale.unflatten(0, (-1, page)).transpose(1, 2).contiguous()
                rows = rows / torch.where(s == 0, 1.0, s)[..., None]
            cache[st["slots"][:real]] = rows
            out[name] = cache.unflatten(0, (-1, page)).transpose(1, 2).contiguous()
        return out
    o = torch.zeros(case["batch"], hq, d, dtype=f, device=DEVICE)
    lse = torch.full((case["batch"], hq), -math.inf, dtype=f, device=DEVICE)
    for i, n in enumerate(st["seq_lens"].tolist()):
        if n == 0:
            continue
        low = max(0, n - case["window"]) if case["window"] else 0
        pages = st["block_table"][i, : -(-n // page)].long()

        def rows(name):
            x = st[name + "_cache"][pages].transpose(0, 1).flatten(1, 2)[:, low:n]
            if case["cache"] == "bf16":
                return x.to(f)
            s = st[name + "_scale"][pages].transpose(0, 1).flatten(1, 2)[:, low:n]
            return x.view(torch.float8_e4m3fn).to(f) * s[..., None].to(f)

        score = st["q"][i].to(f).view(hkv, hq // hkv, d) @ rows("k").transpose(1, 2).contiguous() * d ** -0.5
        if case["softcap"]:
            score = case["softcap"] * torch.tanh(score / case["softcap"])
        lse[i] = torch.logsumexp(score, -1).flatten()
        o[i] = (torch.softmax(score, -1) @ rows("v")).reshape(hq, d)
    return {"o": o, "lse": lse}
