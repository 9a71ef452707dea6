"""examples/decode_layer.py against the layer computed plainly in fp32 from the
dequantized weights.  The library quantizes four activations of the layer and the
cache to e4m3; a code is within 2^-4 of its value, 2.6 % in the root mean square
over uniformly placed mantissas, so each product of independent terms carries about
that much noise.  The largest of the chain's (output projection, gate and up, down,
on top of the attention's) add up to sqrt(5) 2.6 % = 6 %; twice that is asked for."""
from __future__ import annotations

import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


def dense(w):
    codes, scales = w
    n, k = codes.shape
    v = codes.view(torch.float8_e4m3fn).float().view(n // 128, 128, k // 128, 128)
    return (v * scales[:, None, :, None]).reshape(n, k)


def plain_norm(x, gain, eps):
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + eps) * gain.float()


def turn(x, cos_sin, position):
    half = x.shape[-1] // 2
    c, s = cos_sin[position][:, None, :half], cos_sin[position][:, None, half:]
    a, b = x[..., :half], x[..., half:]
    return torch.cat([a * c - b * s, b * c + a * s], -1)


@pytest.mark.parametrize("batch,lengths", [(1, [70]), (3, [5, 200, 131]), (66, [9] * 66)])
def test_layer_steps(gpu_lib, batch, lengths):
    import decode_layer

    torch.manual_seed(1)
    width, hq, hkv, d, hidden = 512, 4, 2, 128, 1024
    layer = decode_layer.DecoderLayer(width, hq, hkv, d, hidden, max_pos=300, seed=2)
    cache = decode_layer.PagedCache(batch, 300, hkv, d, page=32)
    prompt = torch.randn(sum(lengths), width, device="cuda").bfloat16()
    layer.prefill(prompt, cache, lengths)
    wqkv, wout, wgu, wdown = (dense(w) for w in (layer.qkv, layer.out, layer.gate_up, layer.down))

    def project(x, position):  # queries, keys, values of rows x, plainly
        y = (x @ wqkv.t()).view(len(x), hq + 2 * hkv, d)
        return turn(y[:, :hq], layer.cos_sin, position), turn(y[:, hq : hq + hkv], layer.cos_sin, position), y[:, hq + hkv :]

    past, at = [], 0
    for n in lengths:
        x = prompt[at : at + n].float()
        _, k, v = project(plain_norm(x, layer.norm1, layer.eps), torch.arange(n, device="cuda"))
        past.append((k, v))
        at += n
    residual = torch.randn(batch, width, device="cuda").bfloat16()
    stream = residual.float()
    x = torch.randn(batch, width, device="cuda").bfloat16()
    for _ in range(3):
        position, slots = cache.next_slots()
        got = layer.step(x, residual, cache, position, slots)
        stream = stream + x.float()
        q, k, v = project(plain_norm(stream, layer.norm1, layer.eps), position.long())
        rows = []
        for b in range(batch):
            past[b] = (torch.cat([past[b][0], k[b : b + 1]]), torch.cat([past[b][1], v[b : b + 1]]))
            kb, vb = (t.repeat_interleave(hq // hkv, 1).transpose(0, 1).contiguous() for t in past[b])
            p = torch.softmax((kb @ q[b, :, :, None])[..., 0] / d ** 0.5, -1)
            rows.append((p[:, None] @ vb).reshape(-1))
        stream = stream + torch.stack(rows) @ wout.t()
        gate, up = (plain_norm(stream, layer.norm2, layer.eps) @ wgu.t()).chunk(2, -1)
        want = (torch.nn.functional.silu(gate) * up) @ wdown.t()
        torch.cuda.synchronize()
        assert ((residual.float() - stream).norm() / stream.norm()).item() < 0.12
        assert ((got.float() - want).norm() / want.norm()).item() < 0.12
        stream = residual.float()  # the bf16 stream carries on
        x = got
