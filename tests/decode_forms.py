"""Batches that reach each form of the attention's launch plan on a device of 256
compute units: test_decode_plan_cpu.py holds them to their forms, and
test_decode_forms_gpu.py runs them.  Test infrastructure."""
from __future__ import annotations

from typing import NamedTuple

import numpy as np


class Batch(NamedTuple):
    form: tuple  # ("shares", "listed by row" or "by share"), or ("rows", waves of a workgroup, whether divided)
    B: int
    Hq: int
    Hkv: int
    D: int
    page: int
    window: int
    max_len: int

    @property
    def name(self):
        return (f"{'-'.join(str(x) for x in self.form)}-{self.B}x{self.Hq}of{self.Hkv}x{self.D}"
                + (f"-window{self.window}" if self.window else ""))

    def lens(self):
        """Short and empty sequences, and a few on both sides of what the plan turns on."""
        r = np.random.default_rng([self.B, self.Hq, self.D, self.window, self.max_len])
        short = min(90, self.max_len)
        lens = np.where(r.random(self.B) < 0.2, 0, r.integers(0, short + 1, self.B))
        w = self.window or self.max_len - 17
        edges = [n for n in (w - 1, w, w + 1, w + 15, w + 16, w + 17, self.max_len) if 0 <= n <= self.max_len]
        if self.max_len > 1000 and not self.window:
            edges = [1, 33, 700, 1025]
        lens[r.permutation(self.B)[: len(edges)]] = edges[: self.B]
        return [int(n) for n in lens]


ROW, SHARE = ("shares", "listed by row"), ("shares", "by share")
BATCHES = [
    # even shares of more rows than shares
    Batch(SHARE, 260, 32, 8, 128, 16, 0, 4096),
    Batch(SHARE, 300, 24, 8, 64, 48, 0, 4096),
    Batch(SHARE, 131, 8, 8, 256, 32, 0, 4096),
    Batch(SHARE, 1030, 40, 2, 128, 16, 0, 2048),
    Batch(SHARE, 2050, 17, 1, 64, 16, 0, 4096),
    # even shares of windows, both ways of listing the divided rows
    Batch(ROW, 66, 16, 16, 64, 48, 2900, 3000),
    Batch(ROW, 260, 8, 4, 128, 16, 2900, 4096),
    Batch(ROW, 40, 12, 4, 256, 32, 6600, 6800),
    Batch(ROW, 400, 40, 2, 64, 16, 2900, 1 << 17),
    Batch(SHARE, 260, 16, 8, 128, 16, 1701, 3000),
    Batch(SHARE, 300, 8, 8, 64, 64, 2900, 4096),
    Batch(SHARE, 1030, 36, 2, 128, 16, 1701, 3000),
    Batch(SHARE, 131, 24, 8, 256, 16, 1201, 4096),
    # rows of a tile or a few, in workgroups of one, two and four waves
    Batch(("rows", 1, False), 300, 7, 1, 64, 16, 0, 32),
    Batch(("rows", 1, False), 300, 5, 5, 256, 16, 0, 32),
    Batch(("rows", 2, False), 9, 7, 1, 64, 16, 0, 64),
    Batch(("rows", 2, False), 12, 28, 4, 128, 16, 0, 64),
    Batch(("rows", 2, False), 12, 9, 3, 256, 32, 0, 64),
    Batch(("rows", 2, False), 300, 3, 1, 64, 48, 0, 96),
    Batch(("rows", 2, False), 140, 10, 2, 256, 16, 0, 96),
    Batch(("rows", 2, False), 11, 20, 1, 64, 16, 0, 32),
    Batch(("rows", 2, False), 11, 50, 2, 128, 16, 0, 32),
    Batch(("rows", 2, False), 300, 33, 1, 128, 16, 17, 4096),
    Batch(("rows", 2, False), 20, 6, 2, 128, 16, 33, 4096),
    Batch(("rows", 4, False), 9, 15, 3, 64, 16, 0, 96),
    Batch(("rows", 4, False), 9, 36, 2, 128, 16, 0, 64),
    Batch(("rows", 4, False), 9, 5, 1, 256, 16, 50, 4096),
]
