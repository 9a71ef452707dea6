"""Measured cases of the operators that serve prompts and chunks of several tokens.

Three operators, each with its plain form (elementary torch operations in 32 bits, rounded once at the end) and with
the library's call:

* ``append``: root-mean-square norms of the query and key heads of a QKV projection, their rotary position embedding,
  and the append of keys and values to a paged cache (bf16, or e4m3 with one scale for each token and head); on request
  the turned keys in bf16 too;
* ``prompt``: attention over whole prompts of different lengths, packed one behind the other, with grouped heads;
* ``chunk``: attention of the last few or many tokens of each sequence over the paged cache that holds them.

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
MAX_POSITION = 16384  # rows of the rotation table
DEVICE = "cuda"


def listed():
    return [
        # one decoded token: latency of norm, rotation and append
        dict(name="append_token", op="append", tokens=1, padded=0, prompts=1, q_heads=32, kv_heads=8, head_dim=128,
             rotated=128, interleaved=False, page=16, cache="bf16", keys=False),
        # a decode batch padded to 64 rows, into an e4m3 cache
        dict(name="append_batch", op="append", tokens=64, padded=7, prompts=57, q_heads=32, kv_heads=8, head_dim=128,
             rotated=128, interleaved=False, page=64, cache="e4m3", keys=False),
        # three packed prompts of odd lengths, neighbouring pairs rotated in half of each 64-wide head, keys kept for
        # the prompts' own attention
        dict(name="append_prompts", op="append", tokens=4093, padded=0, prompts=3, q_heads=28, kv_heads=4,
             head_dim=64, rotated=32, interleaved=True, page=48, cache="bf16", keys=True),
        # a long prefill into an e4m3 cache, keys kept in bf16 for the prompts' own attention
        dict(name="append_prefill", op="append", tokens=8192, padded=0, prompts=4, q_heads=32, kv_heads=8,
             head_dim=128, rotated=128, interleaved=False, page=16, cache="e4m3", keys=True),
        # a short question: latency
        dict(name="prompt_short", op="prompt", batch=1, shortest=77, longest=77, q_heads=32, kv_heads=8, head_dim=128,
             causal=True, window=0, softcap=0.0),
        # a batch of packed prompts of odd lengths, 64-wide heads
        dict(name="prompt_packed", op="prompt", batch=7, shortest=131, longest=1357, q_heads=28, kv_heads=4,
             head_dim=64, causal=True, window=0, softcap=0.0),
        # one long document
        dict(name="prompt_long", op="prompt", batch=1, shortest=8192, longest=8192, q_heads=32, kv_heads=8,
             head_dim=128, causal=True, window=0, softcap=0.0),
        # 256-wide heads, a sliding window and capped scores
        dict(name="prompt_window", op="prompt", batch=2, shortest=2001, longest=4097, q_heads=16, kv_heads=8,
             head_dim=256, causal=True, window=1024, softcap=30.0),
        # a follow-up of a few tokens on one user's short cache: latency
        dict(name="chunk_short", op="chunk", batch=1, new=7, mixed=False, empty=0, shortest=777, longest=777,
             q_heads=32, kv_heads=8, head_dim=128, page=16, cache="bf16", window=0, softcap=0.0),
        # drafted tokens of a serving batch of ragged lengths, checked over an e4m3 cache
        dict(name="chunk_draft", op="chunk", batch=32, new=4, mixed=False, empty=0, shortest=5, longest=8192,
             q_heads=32, kv_heads=8, head_dim=128, page=64, cache="e4m3", window=0, softcap=0.0),
        # a part of a prompt beside decoding sequences
        dict(name="chunk_mixed", op="chunk", batch=24, new=512, mixed=True, empty=0, shortest=300, longest=4096,
             q_heads=32, kv_heads=8, head_dim=128, page=64, cache="e4m3", window=0, softcap=0.0),
        # a part of a very long prompt behind what is cached of it
        dict(name="chunk_long", op="chunk", batch=1, new=2048, mixed=False, empty=0, shortest=32768, longest=32768,
             q_heads=32, kv_heads=8, head_dim=128, page=16, cache="bf16", window=0, softcap=0.0),
    ]


def _spread(rng, low, high):
    """A whole number of [low, high], spread over its logarithm."""
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


HEADS = [(32, 8), (28, 4), (16, 16), (16, 1), (40, 8), (64, 8), (6, 2), (10, 10), (32, 1)]
PAGES = [16, 32, 48, 64, 128]
MOST_FLOPS = 2 ** 39  # of a drawn attention; the longest listed one has twice that
MOST_SCORES = 2 ** 31  # of its plain form, which pads every sequence to the longest
MOST_CACHED = 2 ** 29  # values of a drawn cache's keys, padded likewise


def draw(rng):
    op = rng.choice(["append", "prompt", "chunk"])
    q_heads, kv_heads = rng.choice(HEADS)
    head_dim = rng.choice([64, 128, 128, 256])
    window, softcap = rng.choice([0, 0, _spread(rng, 1, 4096)]), rng.choice([0.0, 0.0, 30.0])
    shape = dict(op=op, q_heads=q_heads, kv_heads=kv_heads, head_dim=head_dim)
    if op == "append":
        most = 8192 * 48 * 128 // ((q_heads + 2 * kv_heads) * head_dim)
        tokens = _spread(rng, 1, most)
        prompts = tokens if rng.random() < 0.4 and tokens <= 256 else min(tokens, rng.randint(1, 5))
        padded = rng.randint(0, (tokens - prompts) // 8) if tokens > prompts else 0
        return dict(shape, tokens=tokens, padded=padded, prompts=prompts,
                    rotated=rng.choice([head_dim, head_dim, head_dim // 2]), interleaved=rng.random() < 0.4,
                    page=rng.choice(PAGES), cache=rng.choice(["bf16", "e4m3"]), keys=rng.random() < 0.4)
    if op == "prompt":
        batch = _spread(rng, 1, 64)
        most = math.isqrt(min(MOST_SCORES, MOST_FLOPS // (4 * head_dim)) // (batch * q_heads))
        longest = _spread(rng, 1, min(most, 8192))
        causal = rng.random() < 0.8
        return dict(shape, batch=batch, shortest=max(1, int(longest * rng.random())), longest=longest, causal=causal,
                    window=window if causal else 0, softcap=softcap)
    batch = _spread(rng, 1, 64)
    most = min(MOST_SCORES, MOST_FLOPS // (4 * head_dim)) // (batch * q_heads)  # pairs of a new and a cached token
    new = _spread(rng, 1, min(2048, math.isqrt(most)))
    longest = _spread(rng, new, max(new, min(most // new, 32768, MOST_CACHED // (batch * kv_heads * head_dim))))
    return dict(shape, batch=batch, new=new, mixed=rng.random() < 0.3, empty=rng.randint(0, batch // 8),
                shortest=max(1, int(longest * rng.random())), longest=longest, page=rng.choice(PAGES),
                cache=rng.choice(["bf16", "e4m3"]), window=window, softcap=softcap)


def _lengths(case):
    """The sequences' lengths, in order, crowding near the shortest."""
    n = case["batch"]
    u = np.linspace(0.0, 1.0, n) if n > 1 else np.ones(n)
    return case["shortest"] + np.rint((case["longest"] - case["shortest"]) * u * u).astype(np.int64)


def _chunks(case):
    """(new tokens, tokens in the cache) of each sequence: the longest has `new` of them and the others as many, or
    one; the last `empty` of the shorter ones have none in this call."""
    lens = _lengths(case)
    new = np.full(case["batch"], 1 if case["mixed"] else case["new"], dtype=np.int64)
    new[-1] = case["new"]
    new[: case["empty"]] = 0
    return new, np.maximum(lens, new)


def _pairs(new, lens, window, causal=True):
    """Pairs of a query and a key that it sees, summed over the sequences."""
    if not causal:
        return int((new * lens).sum())
    total = 0
    for n, l in zip(new.tolist(), lens.tolist()):
        seen = np.arange(l - n + 1, l + 1)
        total += int((np.minimum(seen, window) if window else seen).sum())
    return total


def work(case):
    hq, hkv, d = case["q_heads"], case["kv_heads"], case["head_dim"]
    if case["op"] == "prompt":
        lens = _lengths(case)
        t = int(lens.sum())
        return {"bytes": t * (hq * (d * 4 + 4) + hkv * d * 4) + 4 * (case["batch"] + 1),
                "flops": _pairs(lens, lens, case["window"], case["causal"]) * hq * d * 4}
    size = 2 if case["cache"] == "bf16" else 1 + 4 / d
    if case["op"] == "append":
        t, stored = case["tokens"], case["tokens"] - case["padded"]
        moved = t * (hq + 2 * hkv) * d * 2 + t * hq * d * 2 + stored * 2 * hkv * d * size + t * 12 + 4 * d
        moved += t * hkv * d * 2 if case["keys"] else 0
        return {"bytes": moved + min(t, MAX_POSITION) * case["rotated"] * 4, "flops": t * (hq + hkv) * d * 10}
    new, lens = _chunks(case)
    window = case["window"]
    read = np.where(new > 0, np.minimum(lens, window + new - 1) if window else lens, 0)
    t = int(new.sum())
    table = int(np.ceil(read / case["page"]).sum()) * 4
    return {"bytes": int(read.sum()) * hkv * d * 2 * size + t * hq * (d * 4 + 4) + table + 8 * case["batch"] + 4,
            "flops": _pairs(new, lens, window) * hq * d * 4}


def _generator(seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(int(seed) * 7919 + 29)
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
    return {"append": _prepare_append, "prompt": _prepare_prompt, "chunk": _prepare_chunk}[case["op"]](case, g, st)


def _prepare_append(case, g, st):
    hq, hkv, d, page = case["q_heads"], case["kv_heads"], case["head_dim"], case["page"]
    t, r = case["tokens"], case["rotated"]
    real, n = t - case["padded"], case["prompts"]
    sizes = torch.full((n,), real // n, dtype=torch.int64)
    sizes[: real % n] += 1
    sizes = sizes.to(DEVICE)
    start = (torch.rand(n, generator=g, device=DEVICE) * (MAX_POSITION - sizes).clamp(min=1)).long()
    prompt = torch.repeat_interleave(torch.arange(n, device=DEVICE), sizes, output_size=real)
    inside = torch.arange(real, device=DEVICE) - (torch.cumsum(sizes, 0) - sizes)[prompt]
    position = (start[prompt] + inside).clamp(max=MAX_POSITION - 1)
    pages = real // page + 2 * n + 1
    order = torch.randperm(pages, generator=g, device=DEVICE)
    held = sizes // page + 2  # pages of each prompt, at most
    local = (start[prompt] + inside) // page - (start // page)[prompt]
    slot = order[(torch.cumsum(held, 0) - held)[prompt] + local] * page + (start[prompt] + inside) % page
    st["qkv"] = _normal(g, t, (hq + 2 * hkv) * d).bfloat16()
    st["q_weight"] = (1.0 + 0.2 * _normal(g, d)).bfloat16()
    st["k_weight"] = (1.0 + 0.2 * _normal(g, d)).bfloat16()
    st["eps"] = 1e-6
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


def _shuffled(n, g):
    return torch.randperm(n, generator=torch.Generator().manual_seed(g.initial_seed())).numpy()


def _starts(counts):
    return torch.from_numpy(np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)).to(DEVICE)


def _prepare_prompt(case, g, st):
    """Queries and turned keys as the append call leaves them, values where the QKV projection left them."""
    hq, hkv, d = case["q_heads"], case["kv_heads"], case["head_dim"]
    lens = _lengths(case)[_shuffled(case["batch"], g)]
    t = int(lens.sum())
    st["counts"], st["starts"] = lens.tolist(), _starts(lens)
    st["q"] = (1.5 * _normal(g, t, hq, d)).bfloat16()
    st["k"] = _normal(g, t, hkv, d).bfloat16()
    qkv = torch.randn(t, hq + 2 * hkv, d, generator=g, device=DEVICE, dtype=torch.bfloat16)
    st["v"] = qkv[:, hq + hkv :]
    return st


def _prepare_chunk(case, g, st):
    hq, hkv, d, page = case["q_heads"], case["kv_heads"], case["head_dim"], case["page"]
    new, lens = _chunks(case)
    order = _shuffled(case["batch"], g)
    new, lens = new[order], lens[order]
    per = torch.from_numpy(-(-lens // page)).to(DEVICE)
    widest, total = int(-(-lens.max() // page)), int((-(-lens // page)).sum()) + 3
    pages = torch.randperm(total, generator=g, device=DEVICE)
    at = (torch.cumsum(per, 0) - per)[:, None] + torch.arange(widest, device=DEVICE)
    used = torch.arange(widest, device=DEVICE) < per[:, None]
    st["block_table"] = torch.where(used, pages[torch.where(used, at, 0)], 0).int()
    st["seq_lens"] = torch.from_numpy(lens.astype(np.int32)).to(DEVICE)
    st["counts"], st["starts"], st["most"] = new.tolist(), _starts(new), int(lens.max())
    st["q"] = (1.5 * _normal(g, int(new.sum()), hq, d)).bfloat16()
    for name in ("k", "v"):
        x = torch.randn(total, hkv, page, d, generator=g, device=DEVICE, dtype=torch.bfloat16)
        if case["cache"] == "bf16":
            st[name + "_cache"] = x
        else:
            st[name + "_cache"], st[name + "_scale"] = _to_cache(x)
        del x
    return st


def run(st):
    return {"append": _append, "prompt": _prompt, "chunk": _chunk}[st["op"]](st)


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
    k = None
    if own:
        import sparse_gemm_linears_amd as sgl
        first = (st["qkv"], st["q_weight"], st["k_weight"], st["positions"], st["slots"], st["cos_sin"])
        more = dict(eps=st["eps"], interleaved=st["interleaved"], return_keys=st["keys"])
        if narrow:
            q = sgl.kv_norm_rope_append_fp8(*first, st["k_cache"], st["v_cache"], st["k_scale"], st["v_scale"], **more)
        else:
            q = sgl.kv_norm_rope_append(*first, st["k_cache"], st["v_cache"], **more)
        if st["keys"]:
            q, k = q
    else:
        t, page, real = st["tokens"], st["page"], st["tokens"] - st["padded"]
        x = st["qkv"].float().view(t, hq + 2 * hkv, -1)
        heads = x[:, : hq + hkv]
        heads = heads * torch.rsqrt((heads * heads).mean(-1, keepdim=True) + st["eps"])
        heads = torch.cat([heads[:, :hq] * st["q_weight"].float(), heads[:, hq:] * st["k_weight"].float()], 1)
        table = st["cos_sin"][st["positions"].long()][:, None]
        turned = _rotate(heads, table[..., : r // 2], table[..., r // 2 :], r, st["interleaved"])
        q = turned[:, :hq].bfloat16()
        if st["keys"]:
            k = turned[:, hq:].bfloat16()
        at, off = st["slots"][:real] // page, st["slots"][:real] % page
        for name, rows in (("k", turned[:real, hq:]), ("v", x[:real, hq + hkv :])):
            if narrow:
                codes, s = _to_cache(rows)
                st[name + "_cache"][at, :, off] = codes
                st[name + "_scale"][at, :, off] = s
            else:
                st[name + "_cache"][at, :, off] = rows.bfloat16()
    out = {"q": q, "keys": k}
    if not narrow:
        return dict(out, k=st["k_cache"], v=st["v_cache"])
    return dict(out, k=st["k_cache"].view(torch.float8_e4m3fn), v=st["v_cache"].view(torch.float8_e4m3fn),
                k_scale=st["k_scale"], v_scale=st["v_scale"])


def _plain_attention(q, k, v, places, lens, st, causal=True):
    """q [B, n, Hq, D] at places [B, n] of their sequences (below 0: no query), k and v [B, Hkv, m, D], of which
    lens [B] count; (o, lse) of [B, n, Hq, ..]."""
    b, n, hq, d = q.shape
    hkv = k.shape[1]
    at = torch.arange(k.shape[2], device=DEVICE)
    live = (at < lens[:, None])[:, None] & (places >= 0)[..., None]  # [B, n, m]
    if causal:
        live = live & (at <= places[..., None])
    if st["window"]:
        live = live & (at > places[..., None] - st["window"])
    live = live[:, None, None]
    heads = q.float().view(b, n, hkv, hq // hkv, d).permute(0, 2, 3, 1, 4).reshape(b, hkv, -1, d)
    score = torch.matmul(heads, k.transpose(-1, -2).contiguous()) * d ** -0.5
    if st["softcap"]:
        score = st["softcap"] * torch.tanh(score / st["softcap"])
    score = score.view(b, hkv, hq // hkv, n, -1).masked_fill(~live, -math.inf)
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - torch.where(torch.isfinite(top), top, 0.0))
    del score
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(b, hkv, -1, p.shape[-1]), v).view(b, hkv, hq // hkv, n, d)
    o = o / torch.where(total == 0, 1.0, total)
    lse = torch.where(total == 0, -math.inf, top + torch.log(total))[..., 0]
    return o.permute(0, 3, 1, 2, 4).reshape(b, n, hq, d).bfloat16(), lse.permute(0, 3, 1, 2).reshape(b, n, hq)


def _places(st):
    """Rows of packed tokens as [B, most]: their numbers, and whether there is one."""
    starts = st["starts"].long()
    at = starts[:-1, None] + torch.arange(max(st["counts"]), device=DEVICE)
    there = at < starts[1:, None]
    return torch.where(there, at, 0), there


def _prompt(st):
    if own:
        import sparse_gemm_linears_amd as sgl
        o, lse = sgl.prompt_attention(st["q"], st["k"], st["v"], st["starts"], softcap=st["softcap"],
                                      window=st["window"], causal=st["causal"], return_lse=True)
        return {"o": o, "lse": lse}
    rows, there = _places(st)
    lens = there.sum(-1)
    place = torch.where(there, torch.arange(rows.shape[1], device=DEVICE), -1)
    k, v = (st[name][rows].float().transpose(1, 2).contiguous() for name in ("k", "v"))
    o, lse = _plain_attention(st["q"][rows], k, v, place, lens, st, st["causal"])
    return {"o": o[there], "lse": lse[there]}


def _chunk(st):
    narrow = st["cache"] == "e4m3"
    if own:
        import sparse_gemm_linears_amd as sgl
        more = dict(softcap=st["softcap"], window=st["window"], max_len=st["most"], return_lse=True)
        if narrow:
            o, lse = sgl.paged_chunk_attention_fp8(st["q"], st["k_cache"], st["v_cache"], st["k_scale"], st["v_scale"],
                                                   st["block_table"], st["seq_lens"], st["starts"], **more)
        else:
            o, lse = sgl.paged_chunk_attention(st["q"], st["k_cache"], st["v_cache"], st["block_table"],
                                               st["seq_lens"], st["starts"], **more)
        return {"o": o, "lse": lse}
    table, d = st["block_table"].long(), st["head_dim"]

    def lines(name):
        x = st[name + "_cache"][table]  # [batch, pages, kv heads, page, d]
        x = x.view(torch.float8_e4m3fn).float() * st[name + "_scale"][table][..., None] if narrow else x.float()
        return x.transpose(1, 2).reshape(x.shape[0], x.shape[2], -1, d)

    rows, there = _places(st)
    lens = st["seq_lens"].long()
    place = lens[:, None] - there.sum(-1, keepdim=True) + torch.arange(rows.shape[1], device=DEVICE)
    o, lse = _plain_attention(st["q"][rows], lines("k"), lines("v"), torch.where(there, place, -1), lens, st)
    return {"o": o[there], "lse": lse[there]}


def exact(case, seed):
    """The outputs in 64 bits.  Codes are given as the quotients that they round, so an error is the rounding's own."""
    st = prepare(case, seed)
    f = torch.float64
    hq, hkv, d = case["q_heads"], case["kv_heads"], case["head_dim"]
    if case["op"] == "append":
        t, r, real, page = case["tokens"], case["rotated"], case["tokens"] - case["padded"], case["page"]
        half = r // 2
        first = torch.arange(half, device=DEVICE) * (2 if case["interleaved"] else 1)
        second = first + (1 if case["interleaved"] else half)
        x = st["qkv"].to(f).view(t, hq + 2 * hkv, d)
        size = torch.linalg.vector_norm(x[:, : hq + hkv], dim=-1) ** 2 / d
        x[:, : hq + hkv] /= torch.sqrt(size + st["eps"])[..., None]
        x[:, :hq] *= st["q_weight"].to(f)
        x[:, hq : hq + hkv] *= st["k_weight"].to(f)
        cs = st["cos_sin"].to(f)[st["positions"].long()]
        turn = torch.complex(cs[:, :half], cs[:, half:])[:, None]
        z = torch.complex(x[..., first], x[..., second])[:, : hq + hkv] * turn
        x[:, : hq + hkv, first], x[:, : hq + hkv, second] = z.real, z.imag
        out = {"q": x[:, :hq], "keys": x[:, hq : hq + hkv] if case["keys"] else None}
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
    o = torch.zeros(st["q"].shape, dtype=f, device=DEVICE)
    lse = torch.full(st["q"].shape[:2], -math.inf, dtype=f, device=DEVICE)
    group, begin = hq // hkv, 0
    for i, n in enumerate(st["counts"]):
        if n == 0:
            continue
        if case["op"] == "prompt":
            length = n
            kv = [st[name][begin : begin + n].to(f).transpose(0, 1) for name in ("k", "v")]
        else:
            length, page = int(st["seq_lens"][i]), case["page"]
            pages = st["block_table"][i, : -(-length // page)].long()
            kv = []
            for name in ("k", "v"):
                x = st[name + "_cache"][pages].transpose(0, 1).flatten(1, 2)[:, :length]
                if case["cache"] == "e4m3":
                    s = st[name + "_scale"][pages].transpose(0, 1).flatten(1, 2)[:, :length]
                    x = x.view(torch.float8_e4m3fn).to(f) * s[..., None].to(f)
                kv.append(x.to(f))
        place = torch.arange(length - n, length, device=DEVICE)[:, None]
        token = torch.arange(length, device=DEVICE)[None]
        hidden = torch.zeros(n, length, dtype=torch.bool, device=DEVICE)
        if case.get("causal", True):
            hidden |= token > place
        if case["window"]:
            hidden |= token <= place - case["window"]
        for h in range(hq):
            keys, values = kv[0][h // group], kv[1][h // group]
            score = st["q"][begin : begin + n, h].to(f) @ keys.t().contiguous() / math.sqrt(d)
            if case["softcap"]:
                score = case["softcap"] * torch.tanh(score / case["softcap"])
            score.masked_fill_(hidden, -math.inf)
            lse[begin : begin + n, h] = torch.logsumexp(score, -1)
            o[begin : begin + n, h] = torch.softmax(score, -1) @ values
        begin += n
    return {"o": o, "lse": lse}
