"""Plain 64-bit references of the decoder-layer operators (norm, rotary append,
paged decode attention), in numpy, from their definitions.  Test
infrastructure: no code shared with the library."""
from __future__ import annotations

import numpy as np
import torch


def bf16(a) -> torch.Tensor:
    """A CPU bf16 tensor of the values of a (rounded to nearest even)."""
    return torch.as_tensor(np.asarray(a, np.float32)).to(torch.bfloat16)


def f64(t: torch.Tensor) -> np.ndarray:
    return t.detach().cpu().to(torch.float64).numpy()


def e4m3_values(codes: torch.Tensor) -> np.ndarray:
    return codes.detach().cpu().view(torch.float8_e4m3fn).to(torch.float64).numpy()


def e4m3_codes_f32(v: np.ndarray, s: np.ndarray) -> np.ndarray:
    """enc(fp32(v / s)) of fp32 rows v [..., n] with fp32 scales s [...]: an IEEE division, then torch's cast (round
    to nearest even) of the quotient clamped to +-448."""
    s = s[..., None].astype(np.float32)
    q = np.where(s == 0, v, np.divide(v, s, out=np.zeros_like(v), where=s != 0)).astype(np.float32)
    return torch.from_numpy(np.clip(q, -448, 448)).to(torch.float8_e4m3fn).view(torch.uint8).numpy()


def norm(x, res, w, eps):
    """(h, v) in 64 bits."""
    h = x if res is None else x + res
    return h, h / np.sqrt((h * h).mean(-1, keepdims=True) + eps) * w


def rotate(x, cos, sin, rot, interleaved):
    """x [T, heads, D], cos and sin [T, rot/2]; also returns |a| + |b| for each value (an error bound's unit)."""
    y, mag = x.copy(), np.abs(x)
    half = rot // 2
    i = np.arange(half)
    a_at, b_at = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    a, b, c, s = x[..., a_at], x[..., b_at], cos[:, None], sin[:, None]
    y[..., a_at], y[..., b_at] = a * c - b * s, b * c + a * s
    mag[..., a_at] = mag[..., b_at] = np.abs(a) + np.abs(b)
    return y, mag


def attention(q, k, v, scale, softcap):
    """q [Hq, D], k and v [Hkv, L, D] of the live tokens: (o, lse, sum p |v|, the largest scale sum |q k|)."""
    hq, d = q.shape
    hkv, length = k.shape[:2]
    if length == 0:
        return np.zeros((hq, d)), np.full(hq, -np.inf), np.zeros((hq, d)), 0.0
    g = hq // hkv
    qg = q.reshape(hkv, g, d)
    s = qg @ k.transpose(0, 2, 1) * scale
    size = abs(scale) * float((np.abs(qg) @ np.abs(k).transpose(0, 2, 1)).max())
    if softcap:
        s = softcap * np.tanh(s / softcap)
    top = s.max(-1, keepdims=True)
    p = np.exp(s - top)
    total = p.sum(-1, keepdims=True)
    p /= total
    return ((p @ v).reshape(hq, d), (top + np.log(total)).reshape(hq), (p @ np.abs(v)).reshape(hq, d), size)
