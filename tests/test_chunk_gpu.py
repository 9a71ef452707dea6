"""paged_chunk_attention and its e4m3 form against the 64-bit reference (tolerances in prompt_ref.py)."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import layer_ref as ref
from prompt_ref import Check
from test_graph_gpu import replay_equals_eager
from test_layer_gpu import gen, paged
from test_prompt_gpu import starts_of

pytestmark = pytest.mark.gpu


def chunk_inputs(new, lens, Hq, Hkv, D, page, fp8, window=0, max_len=None, sharp=1.5, pages=None):
    """Queries, a cache in which everything that no token sees is NaN, and its table; the keys and values that a
    sequence's tokens see in 64 bits, from the first of them on."""
    r = gen("chunk", sum(lens), sum(new), len(lens), Hq, Hkv, D, page, window)
    # the first token of a chunk sees window - 1 keys before it
    reach = [window + n - 1 if window and n else 0 for n in new]
    widest = max(reach)
    dev, table, live = paged(r, lens, Hkv, D, page, fp8, widest, pages=pages)
    if window:  # lines of the widest reach are filled: clear what is beyond each sequence's own
        for b, n in enumerate(lens):
            keep = min(n, reach[b])
            live[b] = [x[:, x.shape[1] - keep :] for x in live[b]]
            for t in range(max(0, n - widest), n - keep):
                for i, cleared in enumerate(dev):
                    cleared[int(table[b, t // page]), :, t % page] = 0x7F if fp8 and i < 2 else float("nan")
    if max_len is not None and table.shape[1] * page < max_len:  # a wider table, its entries out of range
        more = -(-max_len // page) - table.shape[1]
        table = torch.cat([table, torch.full((len(lens), more), -9, dtype=torch.int32, device="cuda")], 1)
    return ref.bf16(sharp * r.standard_normal((sum(new), Hq, D))), dev, table, live


def chunk_case(lib, new, lens, Hq, Hkv, D, page, fp8, window=0, softcap=0.0, max_len=None, scale=None, pages=None):
    q, cache, table, live = chunk_inputs(new, lens, Hq, Hkv, D, page, fp8, window, max_len, pages=pages)
    call = lib.paged_chunk_attention_fp8 if fp8 else lib.paged_chunk_attention
    args = (q.cuda(), *cache, table, torch.tensor(lens, dtype=torch.int32, device="cuda"), starts_of(new))
    kw = dict(window=window, softcap=softcap, max_len=max_len, scale=scale)
    print(f"chunk new={new[:8]} lens={lens[:8]} Hq={Hq} Hkv={Hkv} D={D} page={page} fp8={fp8} {kw}", flush=True)
    o, lse = call(*args, **kw, return_lse=True)
    again = call(*args, **kw)
    torch.cuda.synchronize()
    assert torch.equal(o, again)
    check, at = Check(D ** -0.5 if scale is None else scale, softcap), 0
    for b, (n, length) in enumerate(zip(new, lens)):
        rows = slice(at, at + n)
        k, v = live[b]
        if n:
            check.sequence(o[rows], lse[rows], ref.f64(q[rows]), k, v, k.shape[1] - n, window, True,
                           f"of sequence {b}, {n} of {length}")
        at += n
    check.done()
    return o, lse


#              few over many, whole prompts, one token, none, more than there are
NEW = [1, 3, 7, 16, 33, 64, 100, 1, 0, 5, 17, 129, 2, 4]
LENS = [1, 3, 40, 16, 300, 65, 100, 700, 50, 0, 9, 513, 1, 1025]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("Hq,Hkv,D,page", [(32, 8, 128, 16), (28, 4, 64, 48), (16, 1, 256, 32), (3, 3, 128, 64),
                                           (40, 2, 128, 16), (33, 1, 64, 128), (64, 1, 128, 16), (70, 1, 256, 16),
                                           (8, 8, 64, 16), (10, 5, 256, 1024)])
def test_chunk_edges(gpu_lib, Hq, Hkv, D, page, fp8):
    chunk_case(gpu_lib, NEW, LENS, Hq, Hkv, D, page, fp8)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("window,softcap", [(1, 0.0), (16, 0.0), (17, 30.0), (100, 0.0), (256, 5.0), (5000, 0.0),
                                            (0, 30.0)])
def test_chunk_window_and_cap(gpu_lib, window, softcap, fp8):
    chunk_case(gpu_lib, NEW, LENS, 14, 2, 128, 48, fp8, window=window, softcap=softcap)
    chunk_case(gpu_lib, [1, 20, 300], [900, 900, 900], 4, 2, 64, 16, fp8, window=window, softcap=softcap)
    chunk_case(gpu_lib, [1, 20, 150], [700, 900, 200], 2, 1, 256, 32, fp8, window=window, softcap=softcap)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("new,lens,Hq,Hkv,D,page", [
    ([7], [777], 32, 8, 128, 16), ([1], [20001], 8, 2, 128, 16), ([3, 1], [9973, 3], 8, 1, 64, 64),
    ([4] * 4, [5000, 1, 4999, 17], 16, 16, 64, 48), ([200, 1, 2], [3000, 2500, 4000], 4, 2, 128, 64),
    ([2], [8193], 4, 2, 256, 16), ([1], [4097], 1, 1, 128, 4096), ([512] + [1] * 9, [600] + [2000] * 9, 8, 2, 128, 32)])
def test_chunk_long(gpu_lib, new, lens, Hq, Hkv, D, page, fp8):
    chunk_case(gpu_lib, new, lens, Hq, Hkv, D, page, fp8)


@pytest.mark.parametrize("fp8", [False, True])
def test_a_wider_table_and_bound(gpu_lib, fp8):
    """A bound far above the lengths: parts of the division that have no keys."""
    chunk_case(gpu_lib, [3, 40, 1], [30, 500, 0], 8, 2, 128, 16, fp8, max_len=60000)


def test_one_token_is_the_decode_call(gpu_lib):
    """One new token of each sequence: what paged_decode_attention gives, within both calls' roundings."""
    lens = [1, 70, 300, 999]
    q, cache, table, _ = chunk_inputs([1] * 4, lens, 8, 2, 128, 16, False)
    lens_ = torch.tensor(lens, dtype=torch.int32, device="cuda")
    o, lse = gpu_lib.paged_chunk_attention(q.cuda(), *cache, table, lens_, starts_of([1] * 4), return_lse=True)
    o2, lse2 = gpu_lib.paged_decode_attention(q.cuda(), *cache, table, lens_, return_lse=True)
    assert ((o.float() - o2.float()).norm() / o2.float().norm()).item() < 2.0 ** -8
    assert ((lse - lse2).abs() <= 2.0 ** -17).all()


def test_rows_outside_every_sequence_stay(gpu_lib):
    new, lens = [5, 0, 40], [90, 10, 64]
    q, cache, table, _ = chunk_inputs(new, lens, 4, 2, 64, 16, True)
    pad = torch.zeros(9, 4, 64, dtype=torch.bfloat16)
    q = torch.cat([pad, q, pad]).cuda()
    o = torch.full_like(q, 7.0)
    lse = torch.full(q.shape[:2], 7.0, device="cuda")
    lens_ = torch.tensor(lens, dtype=torch.int32, device="cuda")
    gpu_lib.paged_chunk_attention_fp8(q, *cache, table, lens_, starts_of(new, 9), o=o, lse=lse)
    want = gpu_lib.paged_chunk_attention_fp8(q[9:-9], *cache, table, lens_, starts_of(new))
    assert torch.equal(o[9:-9], want)
    for t in (o, lse):
        assert (t[:9] == 7).all() and (t[-9:] == 7).all() and not (t[9:-9] == 7).any()


@pytest.mark.parametrize("fp8", [False, True])
def test_hidden_values_of_a_cache(gpu_lib, fp8):
    """Values and scales that are not finite reach the tokens that see them, and no token before."""
    new, lens, at = [60], [200], 170  # a token of the chunk itself
    q, cache, table, _ = chunk_inputs(new, lens, 4, 2, 128, 16, fp8)
    call = gpu_lib.paged_chunk_attention_fp8 if fp8 else gpu_lib.paged_chunk_attention
    lens_ = torch.tensor(lens, dtype=torch.int32, device="cuda")
    args = (q.cuda(), *cache, table, lens_, starts_of(new))
    want = call(*args)
    page = int(table[0, at // 16])
    # with an e4m3 cache: a NaN code, a NaN scale, an infinite scale
    for bad in (["code", float("nan"), float("inf")] if fp8 else [float("nan"), float("inf"), float("-inf")]):
        changed = cache[3 if fp8 and bad != "code" else 1]
        kept = changed[page, :, at % 16].clone()
        changed[page, :, at % 16] = 0x7F if bad == "code" else bad
        o = call(*args)
        changed[page, :, at % 16] = kept
        before = at - (200 - 60)
        err = (o[:before].float() - want[:before].float()).abs()
        assert (err <= 2.0 ** -7 * want[:before].float().abs() + 2.0 ** -16).all(), bad
        assert not torch.isfinite(o[before:]).any(), bad


def test_bad_pages_are_clamped(gpu_lib):
    """Page numbers out of range: such rows are unspecified, the others keep their results."""
    new, lens = [3, 20, 4], [64, 100, 33]
    q, cache, table, _ = chunk_inputs(new, lens, 4, 2, 64, 16, False)
    lens_ = torch.tensor(lens, dtype=torch.int32, device="cuda")
    want = gpu_lib.paged_chunk_attention(q.cuda(), *cache, table, lens_, starts_of(new))
    bad = table.clone()
    wild = torch.tensor([-1, 1 << 30, -(1 << 31), (1 << 31) - 1] * 2, dtype=torch.int32, device="cuda")
    bad[1] = wild[: bad.shape[1]]
    got = gpu_lib.paged_chunk_attention(q.cuda(), *cache, bad, lens_, starts_of(new))
    assert torch.equal(got[:3], want[:3]) and torch.equal(got[23:], want[23:])


@pytest.mark.parametrize("new,lens", [([4, 1, 2], [700, 3000, 64]), ([64, 1], [300, 900])])
def test_chunk_in_a_graph(gpu_lib, new, lens):
    q, cache, table, _ = chunk_inputs(new, lens, 8, 2, 128, 16, True)
    q, starts = q.cuda(), starts_of(new)
    lens_ = torch.tensor(lens, dtype=torch.int32, device="cuda")
    o, lse = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")
    replay_equals_eager(lambda: gpu_lib.paged_chunk_attention_fp8(q, *cache, table, lens_, starts, o=o, lse=lse),
                        [o, lse])


def test_lengths_change_between_replays(gpu_lib):
    """A captured call reads lengths, starts and pages when it runs."""
    q, cache, table, _ = chunk_inputs([30, 30], [400, 900], 8, 2, 128, 16, False)
    q = q.cuda()
    starts, lens_ = starts_of([30, 30]), torch.tensor([400, 900], dtype=torch.int32, device="cuda")
    o = torch.zeros_like(q)
    call = lambda: gpu_lib.paged_chunk_attention(q, *cache, table, lens_, starts, o=o)  # noqa: E731
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        call()
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for first, lens in ((30, [400, 900]), (1, [17, 900]), (59, [399, 1]), (0, [5, 777])):
        starts.copy_(torch.tensor([0, first, 60], dtype=torch.int32))
        lens_.copy_(torch.tensor(lens, dtype=torch.int32))
        g.replay()
        torch.cuda.synchronize()
        got = o.clone()
        call()
        torch.cuda.synchronize()
        assert torch.equal(got, o), (first, lens)


def test_binding_refusals(gpu_lib):
    q, cache, table, _ = chunk_inputs([3, 2], [9, 20], 4, 2, 64, 16, False)
    q, lens = q.cuda(), torch.tensor([9, 20], dtype=torch.int32, device="cuda")
    starts = starts_of([3, 2])
    f = gpu_lib.paged_chunk_attention
    with pytest.raises(ValueError, match="block_table"):
        f(q, *cache, table[:1], lens, starts)
    with pytest.raises(ValueError, match="seq_lens"):
        f(q, *cache, table, lens[:1], starts)
    with pytest.raises(TypeError, match="starts"):
        f(q, *cache, table, lens, starts.long())
    with pytest.raises(ValueError, match="q:"):
        f(q[..., :32].contiguous(), *cache, table, lens, starts)
    with pytest.raises(TypeError, match="k_cache"):
        gpu_lib.paged_chunk_attention_fp8(q, *cache, cache[0], cache[0], table, lens, starts)
    for bad in (dict(max_len=10 ** 6), dict(max_len=-1), dict(window=-1), dict(scale=float("inf")), dict(softcap=-1.0)):
        with pytest.raises(gpu_lib.Fp8LinError):
            f(q, *cache, table, lens, starts, **bad)


def shared_pages(D, Hkv, length, page, fp8, seed):
    """A cache of one sequence of `length` tokens and its table's row: (cache, row, keys, values in 64 bits)."""
    dev, table, live = paged(gen("shared pages", seed), [length], Hkv, D, page, fp8, 0)
    return dev, table[0], live[0]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("B,new,length,Hq,Hkv,D,page", [
    (300, 1, 4500, 16, 8, 64, 32), (160, 3, 4500, 16, 8, 128, 16), (90, 1, 2300, 16, 16, 256, 64),
    (40, 130, 2300, 8, 4, 128, 48), (70, 40, 1100, 4, 2, 64, 16)])
def test_many_sequences_without_division(gpu_lib, B, new, length, Hq, Hkv, D, page, fp8):
    """Batches that fill the device, so that a workgroup goes over a whole cache (and looks its pages up again and
    again).  The sequences share their pages and stand at other lengths; a few of them are checked."""
    cache, row, (k, v) = shared_pages(D, Hkv, length, page, fp8, B)
    r = gen("filling", B)
    lens = [length - (b * 37) % 200 for b in range(B)]
    q = ref.bf16(1.5 * r.standard_normal((B * new, Hq, D)))
    table = row.expand(B, -1).contiguous()
    lens_ = torch.tensor(lens, dtype=torch.int32, device="cuda")
    call = gpu_lib.paged_chunk_attention_fp8 if fp8 else gpu_lib.paged_chunk_attention
    o, lse = call(q.cuda(), *cache, table, lens_, starts_of([new] * B), return_lse=True)
    check = Check(D ** -0.5, 0.0)
    for b in (0, 1, B // 2, B - 1):
        rows, n = slice(b * new, (b + 1) * new), lens[b]
        check.sequence(o[rows], lse[rows], ref.f64(q[rows]), k[:, :n], v[:, :n], n - new, what=f"of sequence {b}")
    check.done()


@pytest.mark.parametrize("fp8", [False, True])
def test_lines_past_32_bits(gpu_lib, fp8):
    """A cache of more than 2^32 values, its last pages used: offsets that do not fit 32 bits."""
    pages = (1 << 32) // (16 * 8 * 128) + 300
    chunk_case(gpu_lib, [3, 90], [50, 133], 16, 8, 128, 16, fp8, pages=pages)


def test_searches_of_many_sequences(gpu_lib):
    """More sequences than one search round of 64 and of 4096 finds, most of them without tokens."""
    for B in (65, 5000):
        new = [0] * B
        for b in (0, 1, 63, 64, B // 2, B - 1):
            new[b] = 1 + b % 3
        cache, row, (k, v) = shared_pages(64, 1, 40, 16, False, B)
        q = ref.bf16(gen("search", B).standard_normal((sum(new), 2, 64)))
        lens = torch.full((B,), 40, dtype=torch.int32, device="cuda")
        o, lse = gpu_lib.paged_chunk_attention(q.cuda(), *cache, row.expand(B, -1).contiguous(), lens, starts_of(new),
                                               return_lse=True)
        check, at = Check(64 ** -0.5, 0.0), 0
        for b, n in enumerate(new):
            if n:
                rows = slice(at, at + n)
                check.sequence(o[rows], lse[rows], ref.f64(q[rows]), k, v, 40 - n, what=f"of sequence {b}")
            at += n
        check.done()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("B,D,Hkv,group,window", [(2, 128, 2, 4, 0), (63, 64, 1, 2, 0), (65, 128, 1, 16, 0),
                                                  (130, 64, 1, 3, 100), (256, 128, 1, 1, 0), (257, 64, 1, 1, 0),
                                                  (9, 256, 2, 2, 0), (24, 128, 3, 5, 300)])
def test_shares_of_ragged_sequences(gpu_lib, B, D, Hkv, group, window, fp8):
    """Batches of sequences from no key to thousands, single tokens beside long chunks and beside none, divided by
    their lengths."""
    cache, row, (k, v) = shared_pages(D, Hkv, 4096, 32, fp8, B)
    r = gen("shares", B, D)
    lens = [int(4096 ** x) for x in r.random(B)]
    new = [int(x) for x in r.integers(0, 4, B)]
    for b in (0, B // 2, B - 1):  # long ones, a chunk, and an empty one
        lens[b], new[b] = 4096 - b % 7, 1 + 70 * (b == B // 2)
    lens[B // 3], new[B // 3] = (0, 2) if B > 3 else (4096, 1)
    q = ref.bf16(1.5 * r.standard_normal((sum(new), Hkv * group, D)))
    call = gpu_lib.paged_chunk_attention_fp8 if fp8 else gpu_lib.paged_chunk_attention
    table = row.expand(B, -1).contiguous()
    o, lse = call(q.cuda(), *cache, table, torch.tensor(lens, dtype=torch.int32, device="cuda"), starts_of(new),
                  window=window, return_lse=True)
    check, at = Check(D ** -0.5, 0.0), 0
    for b, n in enumerate(new):
        rows = slice(at, at + n)
        if n and (lens[b] > 2000 or b % 5 == 0 or n > lens[b]):
            check.sequence(o[rows], lse[rows], ref.f64(q[rows]), k[:, : lens[b]], v[:, : lens[b]], lens[b] - n,
                           window, what=f"of sequence {b}")
        at += n
    check.done()
    again = call(q.cuda(), *cache, table, torch.tensor(lens, dtype=torch.int32, device="cuda"), starts_of(new),
                 window=window)
    assert torch.equal(again, o)  # no order of the parts changes a result


def test_unordered_starts_stay_in_bounds(gpu_lib):
    """Starts that fall, or lie outside the rows: their sequences' rows are unspecified, and a sequence beside them
    whose rows no other one claims keeps its results where it is found."""
    new, lens = [4, 4, 4], [30, 40, 50]
    q, cache, table, _ = chunk_inputs(new, lens, 2, 1, 64, 16, False)
    lens_ = torch.tensor(lens, dtype=torch.int32, device="cuda")
    for bad in ([0, 9, 3, 12], [-5, 4, 8, 400], [12, 8, 4, 0], [1 << 30, -(1 << 31), (1 << 31) - 1, 5]):
        starts = torch.tensor(bad, dtype=torch.int32, device="cuda")
        o = torch.zeros(14, 2, 64, dtype=torch.bfloat16, device="cuda")  # two rows more than there are
        gpu_lib.paged_chunk_attention(q.cuda(), *cache, table, lens_, starts, o=o[:12])
        gpu_lib.prompt_attention(q.cuda(), q[:, :1].cuda(), q[:, :1].cuda(), starts, o=o[:12])
        torch.cuda.synchronize()
        assert (o[12:] == 0).all()


def test_unordered_starts_of_divided_sequences(gpu_lib):
    """Starts that make more rows than there are: no part lies past the partials' memory."""
    T = 300
    cache, row, _ = shared_pages(64, 1, 2000, 16, False, 3)
    q = ref.bf16(gen("unordered").standard_normal((T, 8, 64)))
    for B in (3, 100):
        table = row.expand(B, -1).contiguous()
        lens = torch.full((B,), 2000, dtype=torch.int32, device="cuda")
        for high in (T, 1 << 30):
            starts = torch.tensor([0 if b % 2 else high for b in range(B + 1)], dtype=torch.int32, device="cuda")
            o = torch.zeros(T + 2, 8, 64, dtype=torch.bfloat16, device="cuda")
            gpu_lib.paged_chunk_attention(q.cuda(), *cache, table, lens, starts, o=o[:T])
            torch.cuda.synchronize()
            assert (o[T:] == 0).all()


def test_two_streams_and_two_graphs(gpu_lib):
    """Divided calls at once on two streams, and two graphs of such calls replayed in turn: each has scratch memory of
    its own."""
    cases = []
    for i, (new, lens) in enumerate((([4, 2], [900, 3000]), ([40], [2500]))):
        q, cache, table, _ = chunk_inputs(new, lens, 8, 2, 128, 16, bool(i))
        call = gpu_lib.paged_chunk_attention_fp8 if i else gpu_lib.paged_chunk_attention
        args = (q.cuda(), *cache, table, torch.tensor(lens, dtype=torch.int32, device="cuda"), starts_of(new))
        cases.append((call, args, call(*args), torch.empty_like(args[0])))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    for _ in range(5):
        for s, (call, args, _, o) in zip(streams, cases):
            with torch.cuda.stream(s):
                call(*args, o=o)
    torch.cuda.synchronize()
    assert all(torch.equal(want, o) for _, _, want, o in cases)
    graphs = []
    for s, (call, args, _, o) in zip(streams, cases):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            call(*args, o=o)
        graphs.append(g)
    for _ in range(3):
        for _, _, _, o in cases:
            o.zero_()
        torch.cuda.synchronize()
        for s, g in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(want, o) for _, _, want, o in cases)
        for call, args, want, _ in cases:  # eager work between the replays
            assert torch.equal(call(*args), want)
