"""One decoder layer served on the library's calls alone, prompts first and then a token at a time.

The layer keeps e4m3 weights in 128x128 blocks and a paged e4m3 key-value cache.  A
step takes the batch's residual stream and last block's output and runs

    fp8_add_rmsnorm -> fp8_block_gemm (QKV) -> kv_rope_append_fp8 -> paged_decode_attention_fp8
    -> fp8_block_linear (output projection) -> fp8_add_rmsnorm -> fp8_block_gemm_swiglu -> fp8_block_gemm (down)

so that nothing but the library's kernels runs between two layers.  Whole prompts run
kv_norm_rope_append_fp8 and prompt_attention in the place of the two calls in the middle (their own
keys are still there in bf16), and chunks of tokens behind what is cached kv_norm_rope_append_fp8
and paged_chunk_attention_fp8.  Run as a program (on an MI355X) it passes a prompt
through the layer, whole and in chunks, decodes a few tokens with the sizes of a
Llama-3-8B layer and random weights, eagerly and as a replayed HIP graph, and prints
the times.
"""
from __future__ import annotations

import argparse
import math
import os
import sys
import time

import torch

if __name__ == "__main__":
    sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import sparse_gemm_linears_amd as sgl


def rotation_table(max_pos: int, rot: int, theta: float = 10000.0, device="cuda") -> torch.Tensor:
    """cos_sin [max_pos, rot] fp32 for kv_rope_append: rot/2 cosines, then rot/2 sines of each position."""
    angle = torch.arange(max_pos, device=device, dtype=torch.float64)[:, None] \
        * theta ** (-torch.arange(0, rot, 2, device=device, dtype=torch.float64) / rot)
    return torch.cat([angle.cos(), angle.sin()], -1).float()


class PagedCache:
    """e4m3 keys and values of a batch of sequences, with pages handed out in any order."""

    def __init__(self, batch, max_len, heads, dim, page=64, device="cuda"):
        self.page, self.per = page, -(-max_len // page)
        pages = batch * self.per
        self.k, self.v = (torch.empty(pages, heads, page, dim, dtype=torch.uint8, device=device) for _ in range(2))
        self.ks, self.vs = (torch.empty(pages, heads, page, dtype=torch.float32, device=device) for _ in range(2))
        self.table = torch.randperm(pages, device=device).view(batch, self.per).int()
        self.lens = torch.zeros(batch, dtype=torch.int32, device=device)
        self.max_len = self.per * page

    def slots(self, sequence, position):
        """Cache lines of tokens: int64 tensors of sequence numbers and positions in them."""
        return self.table[sequence, position // self.page].long() * self.page + position % self.page

    def next_slots(self):
        """Positions and lines of one new token of every sequence; the lengths then count it."""
        position = self.lens.clone()
        slots = self.slots(torch.arange(len(position), device=position.device), position.long())
        self.lens += 1
        return position, slots


class DecoderLayer:
    def __init__(self, width=4096, q_heads=32, kv_heads=8, dim=128, hidden=14336, max_pos=8192, seed=0,
                 device="cuda", head_norms=False):
        g = torch.Generator(device=device).manual_seed(seed)
        self.q_heads, self.kv_heads, self.dim, self.eps = q_heads, kv_heads, dim, 1e-5

        def linear(n, k):
            return sgl.fp8_quant_weight_block((torch.randn(n, k, generator=g, device=device) / math.sqrt(k)).bfloat16())

        def gain():
            return (1 + 0.1 * torch.randn(width, generator=g, device=device)).bfloat16()

        self.norm1, self.norm2 = gain(), gain()
        self.qkv = linear((q_heads + 2 * kv_heads) * dim, width)
        self.out = linear(width, q_heads * dim)
        self.gate_up = linear(2 * hidden, width)
        self.down = linear(width, hidden)
        self.cos_sin = rotation_table(max_pos, dim, device=device)
        # gains of the query and key heads' norms, in layers that have them
        self.head_gains = [None, None]
        if head_norms:
            self.head_gains = [(1 + 0.1 * torch.randn(dim, generator=g, device=device)).bfloat16() for _ in range(2)]

    def prefill(self, x, cache: PagedCache, lengths):
        """Append the keys and values of packed prompts x [T, width] bf16 of the given lengths; the rotated queries."""
        device = x.device
        counts = torch.tensor(lengths, device=device)
        sequence = torch.repeat_interleave(torch.arange(len(lengths), device=device), counts)
        position = torch.arange(len(x), device=device) - (counts.cumsum(0) - counts)[sequence]
        _, _, xq, xs = sgl.fp8_add_rmsnorm(x, self.norm1, eps=self.eps)
        qkv = sgl.fp8_block_gemm(xq, xs, *self.qkv)
        cache.lens.copy_(counts)
        return sgl.kv_rope_append_fp8(qkv, position.int(), cache.slots(sequence, position), self.cos_sin, cache.k,
                                      cache.v, cache.ks, cache.vs)

    def prompts(self, x, residual, cache: PagedCache, lengths):
        """Whole prompts of the given lengths, packed: x [T, width] is added to residual (updated in place); returns the
        output that the next layer adds.  Their keys and values fill the (empty) cache."""
        counts, sequence, starts = self._packed(lengths, x.device)
        position = torch.arange(len(x), device=x.device) - starts[sequence]
        cache.lens.copy_(counts)
        qkv = self._project(x, residual)
        q, k = sgl.kv_norm_rope_append_fp8(qkv, *self.head_gains, position.int(), cache.slots(sequence, position),
                                           self.cos_sin, cache.k, cache.v, cache.ks, cache.vs, eps=self.eps,
                                           return_keys=True)
        v = qkv.view(len(x), -1, self.dim)[:, self.q_heads + self.kv_heads :]  # where the projection left them
        return self._rest(sgl.prompt_attention(q, k, v, starts), residual)

    def chunk(self, x, residual, cache: PagedCache, new):
        """new[b] further tokens of each sequence (none, one or many), packed: as ``prompts``, behind what is cached."""
        counts, sequence, starts = self._packed(new, x.device)
        position = cache.lens[sequence] + torch.arange(len(x), device=x.device) - starts[sequence]
        cache.lens += counts.int()
        q = sgl.kv_norm_rope_append_fp8(self._project(x, residual), *self.head_gains, position.int(),
                                        cache.slots(sequence, position), self.cos_sin, cache.k, cache.v, cache.ks,
                                        cache.vs, eps=self.eps)
        o = sgl.paged_chunk_attention_fp8(q, cache.k, cache.v, cache.ks, cache.vs, cache.table, cache.lens, starts,
                                          max_len=cache.max_len)
        return self._rest(o, residual)

    @staticmethod
    def _packed(lengths, device):
        """Counts, sequence of each token and starts of packed tokens."""
        counts = torch.tensor(lengths, device=device)
        sequence = torch.repeat_interleave(torch.arange(len(lengths), device=device), counts)
        starts = torch.zeros(len(lengths) + 1, dtype=torch.int32, device=device)
        starts[1:] = counts.cumsum(0)
        return counts, sequence, starts

    def _project(self, x, residual):
        _, _, xq, xs = sgl.fp8_add_rmsnorm(x, self.norm1, residual, eps=self.eps, h=residual)
        return sgl.fp8_block_gemm(xq, xs, *self.qkv)

    def step(self, x, residual, cache: PagedCache, position, slots):
        """One token of each sequence: x [B, width] is added to residual (updated in place); returns the output that
        the next layer adds.  cache.lens counts the new token already."""
        qkv = self._project(x, residual)
        if self.head_gains[0] is None:
            q = sgl.kv_rope_append_fp8(qkv, position, slots, self.cos_sin, cache.k, cache.v, cache.ks, cache.vs)
        else:
            q = sgl.kv_norm_rope_append_fp8(qkv, *self.head_gains, position, slots, self.cos_sin, cache.k, cache.v,
                                            cache.ks, cache.vs, eps=self.eps)
        o = sgl.paged_decode_attention_fp8(q, cache.k, cache.v, cache.ks, cache.vs, cache.table, cache.lens,
                                           max_len=cache.max_len)
        return self._rest(o, residual)

    def _rest(self, o, residual):
        """The layer behind its attention's output o [rows, heads, dim]."""
        o = o.view(o.shape[0], self.q_heads * self.dim)
        if o.shape[0] <= sgl.MAX_LINEAR_M:
            a = sgl.fp8_block_linear(o, *self.out)
        else:
            a = sgl.fp8_block_gemm(*sgl.fp8_quant_act(o), *self.out)
        _, _, xq, xs = sgl.fp8_add_rmsnorm(a, self.norm2, residual, eps=self.eps, h=residual)
        _, hq, hs = sgl.fp8_block_gemm_swiglu(xq, xs, *self.gate_up, keep_h=False)
        return sgl.fp8_block_gemm(hq, hs, *self.down)


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--batch", type=int, default=16)
    ap.add_argument("--prompt", type=int, default=1000, help="tokens of each prompt")
    ap.add_argument("--tokens", type=int, default=32, help="tokens to decode for each sequence")
    a = ap.parse_args()
    layer = DecoderLayer(max_pos=a.prompt + 2 * a.tokens + 8)
    cache = PagedCache(a.batch, a.prompt + 2 * a.tokens + 8, layer.kv_heads, layer.dim)
    prompt = torch.randn(a.batch * a.prompt, 4096, device="cuda").bfloat16()
    stream_in = torch.zeros_like(prompt)
    half = a.prompt // 2

    def timed(f):
        f()
        torch.cuda.synchronize()
        begin = time.perf_counter()
        f()
        torch.cuda.synchronize()
        return time.perf_counter() - begin

    def in_chunks():
        cache.lens.zero_()
        for n in (half, a.prompt - half):
            layer.chunk(prompt[: a.batch * n], stream_in[: a.batch * n], cache, [n] * a.batch)

    chunks = timed(in_chunks)
    whole = timed(lambda: layer.prompts(prompt, stream_in, cache, [a.prompt] * a.batch))
    print(f"{a.batch} prompts of {a.prompt} tokens: {whole * 1e3:.2f} ms whole, {chunks * 1e3:.2f} ms in two chunks")
    x = torch.randn(a.batch, 4096, device="cuda").bfloat16()
    residual = torch.zeros_like(x)
    for _ in range(3):
        layer.step(x, residual, cache, *cache.next_slots())
    torch.cuda.synchronize()
    begin = time.perf_counter()
    for _ in range(a.tokens):
        layer.step(x, residual, cache, *cache.next_slots())
    torch.cuda.synchronize()
    eager = (time.perf_counter() - begin) / a.tokens

    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        layer.step(x, residual, cache, *cache.next_slots())
    torch.cuda.current_stream().wait_stream(stream)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer.step(x, residual, cache, *cache.next_slots())
    torch.cuda.synchronize()
    begin = time.perf_counter()
    for _ in range(a.tokens):
        graph.replay()
    torch.cuda.synchronize()
    replayed = (time.perf_counter() - begin) / a.tokens
    print(f"{a.batch} sequences from {a.prompt} tokens on: a layer's step {eager * 1e6:.1f} us eager, "
          f"{replayed * 1e6:.1f} us as a graph")


if __name__ == "__main__":
    main()
