"""Plain 64-bit reference of the attention of several tokens, in numpy, from its
definition, and the tolerances of the library's.  Test infrastructure: no code shared
with the library.

With u = 2^-24 and S the largest sum of scale |q_d k_d| of a sequence, a score is within
(D + 8) u S (plus a cap's tanh: 2^-20 softcap, and 2^-19 of a score).  o is within twice
that, plus 2^-8 for the weights' one bf16 each and u for each key of a chain, times
sum p |v|, before its own rounding; lse within the score's error, 2^-19 and u for each key.

The roundings of the weights are independent: over many values, the squared error is
that of the roundings, uniform in +-2^-8 of a weight and of an output at most, so
2^-16 / 3 of sum p^2 v^2 and of o^2 each; the test asks for twice the root of that (four
times the expected squares) over all values of a call, beside the score's part.
"""
from __future__ import annotations

import numpy as np
import torch

import layer_ref as ref
from test_layer_gpu import U, assert_rounded, holds


def attend(q, k, v, place0, scale, softcap=0.0, window=0, causal=True):
    """q [n, Hq, D] at places place0 .. of the keys k, v [Hkv, L, D]; hidden keys and values may be anything.
    (o, lse, sum p |v|, sum p^2 v^2, S)."""
    n, hq, d = q.shape
    hkv, length = k.shape[:2]
    o, spread, squares = (np.zeros((n, hq, d)) for _ in range(3))
    lse = np.full((n, hq), -np.inf)
    place = place0 + np.arange(n)[:, None]
    token = np.arange(length)[None]
    seen = np.broadcast_to(token <= place if causal else token >= 0, (n, length)).copy()
    if window:
        seen &= token > place - window
    used = seen.any(0)
    if not used.any():
        return o, lse, spread, squares, 0.0
    size = 0.0
    for h in range(hq):
        kh, vh = k[h // (hq // hkv)][used], v[h // (hq // hkv)][used]
        s = q[:, h] @ kh.T * scale
        size = max(size, abs(scale) * float((np.abs(q[:, h]) @ np.abs(kh).T).max()))
        if softcap:
            s = softcap * np.tanh(s / softcap)
        s[~seen[:, used]] = -np.inf
        top = s.max(-1, keepdims=True)
        p = np.exp(s - np.where(np.isfinite(top), top, 0))
        total = p.sum(-1, keepdims=True)
        with np.errstate(divide="ignore"):
            lse[:, h] = np.where(total > 0, top + np.log(total), -np.inf)[:, 0]
        p /= np.where(total > 0, total, 1)
        o[:, h], spread[:, h], squares[:, h] = p @ vh, p @ np.abs(vh), (p * p) @ (vh * vh)
    return o, lse, spread, squares, size


class Check:
    """Holds a call's outputs to the reference, a sequence at a time."""

    def __init__(self, scale, softcap):
        self.scale, self.softcap = scale, softcap
        self.off = self.expected = self.slack = 0.0

    def sequence(self, o, lse, q, k, v, place0, window=0, causal=True, what=""):
        d = q.shape[-1]
        want, want_lse, spread, squares, size = attend(q, k, v, place0, self.scale, self.softcap, window, causal)
        keys = k.shape[1]
        score = (d + 8) * U * size + (min(2.0 ** -20 * self.softcap, 2.0 ** -19 * size) if self.softcap else 0.0)
        assert_rounded(o, want, (2 * score + 2.0 ** -8 * (1 + 2.0 ** -8) + keys * U) * spread, "o " + what)
        lse = ref.f64(lse)
        empty = np.isneginf(want_lse)
        assert np.isneginf(lse[empty]).all() and (ref.f64(o)[empty] == 0).all(), what
        full = ~empty
        holds(np.abs(lse[full] - want_lse[full]) <= score + 2.0 ** -19 + keys * U + 2.0 ** -22 * np.abs(want_lse[full]),
              "lse " + what)
        self.off += float(((ref.f64(o) - want) ** 2).sum())
        self.expected += 2.0 ** -16 / 3 * float(squares.sum() + (want * want).sum())
        self.slack += float(((2 * score + keys * U) * spread).__pow__(2).sum())

    def done(self):
        assert np.sqrt(self.off) <= 2 * np.sqrt(self.expected) + np.sqrt(self.slack), (self.off, self.expected)


def heads(t: torch.Tensor) -> np.ndarray:
    """[tokens, heads, D] as 64-bit [heads, tokens, D]."""
    return ref.f64(t).transpose(1, 0, 2)
