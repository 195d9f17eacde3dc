"""Oracle of the paged cache of the model's own type, and of the appends with rotation.

Plain NumPy from the definitions (include/kvb.h, kvb_paged_append and kvb_paged_attention),
one token and one sequence at a time; attention is the 8-bit cache's over other pages.
"""
from __future__ import annotations

import numpy as np

from .cache8 import Cache8
from .kvb_oracle import inv_freq


def table(theta: float, d: int, max_pos: int):
    """cos and sin [max_pos][d/2], float64 angles, as float32 numbers."""
    angle = np.arange(max_pos, dtype=np.float64)[:, None] * inv_freq(theta, d)[None]
    return np.cos(angle).astype(np.float32), np.sin(angle).astype(np.float32)


def rotate32(x, pos, cos, sin) -> np.ndarray:
    """Rows x [...][T][d] at positions pos [T] in float32, every product and sum rounded by itself; 0 where pos is not in the table."""
    x = np.asarray(x, dtype=np.float32)
    half = x.shape[-1] // 2
    ok = (np.asarray(pos) >= 0) & (np.asarray(pos) < len(cos))
    at = np.where(ok, pos, 0)
    c, s, lo, hi = cos[at], sin[at], x[..., :half], x[..., half:]
    with np.errstate(invalid="ignore", over="ignore"):
        out = np.concatenate([lo * c - hi * s, hi * c + lo * s], axis=-1)
    return np.where(ok[:, None], out, np.float32(0))


class Paged(Cache8):
    """pages k, v [L][n_pages][H][page][d] in float64; attention() as the 8-bit cache's."""

    def __init__(self, L, n_pages, H, page, d):
        self.page = page
        self.codes = [np.full((L, n_pages, H, page, d), np.nan) for _ in range(2)]

    def append(self, kv, x, page_table, seq_off, seq_pos, l_begin=0):
        x = np.asarray(x, dtype=np.float64)
        for s in range(len(seq_pos)):
            for i in range(int(seq_off[s + 1] - seq_off[s])):
                p, t = int(seq_pos[s]) + i, int(seq_off[s]) + i
                self.codes[kv][l_begin:l_begin + x.shape[0], int(page_table[s][p // self.page]), :, p % self.page] = x[:, :, t]

    def sequence(self, kv, page_row, n, l, h):
        ids = np.asarray(page_row[:-(-n // self.page)], dtype=np.int64)
        if n == 0:
            return np.zeros((0, self.codes[kv].shape[4]))
        x = self.codes[kv][l, ids, h]
        return x.reshape(-1, x.shape[-1])[:n]
