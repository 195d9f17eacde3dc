"""Float64 oracle of the paged 8-bit cache: e4m3 codes, one power-of-two scale
for each (layer, page, head) block of K and of V.

Plain NumPy from the definitions (include/kvb.h, kvb_cache8), one block and one
sequence at a time; pinned by tests/test_oracle_cache8.py to what the format
and the mathematics fix.
"""
from __future__ import annotations

import numpy as np

E_MIN, E_MAX, CODE_MAX = -117, 119, 448.0


def e4m3_values() -> np.ndarray:
    """Value of each byte: sign, 4 exponent bits (bias 7), 3 fraction bits; 0x7f and 0xff are NaN."""
    out = np.empty(256)
    for b in range(256):
        e, f = (b >> 3) & 15, b & 7
        v = f * 2.0 ** -9 if e == 0 else (1 + f / 8) * 2.0 ** (e - 7)
        out[b] = np.nan if (b & 127) == 127 else (-v if b & 128 else v)
    return out


_POS = e4m3_values()[:127]  # 0 .. 448, ascending


def e4m3_encode(x) -> np.ndarray:
    """Bytes of x rounded to the nearest e4m3 number, ties to the even byte, saturating at 448; a zero keeps its sign."""
    x = np.asarray(x, dtype=np.float64)
    a = np.minimum(np.abs(x), CODE_MAX)
    hi = np.minimum(np.searchsorted(_POS, a), 126)
    lo = np.maximum(hi - 1, 0)
    up, down = _POS[hi] - a, a - _POS[lo]
    code = np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    return (code | np.where(np.signbit(x), 128, 0)).astype(np.uint8)


def block_exponent(amax: float) -> int:
    """The smallest e in [E_MIN, E_MAX] with amax <= 448 * 2^e."""
    e = E_MIN
    while e < E_MAX and amax > CODE_MAX * 2.0 ** e:
        e += 1
    return e


class Cache8:
    """k, v bytes [L][n_pages][H][page][d]; k_scale, v_scale [L][n_pages][H]."""

    def __init__(self, L, n_pages, H, page, d):
        self.page = page
        self.codes = [np.zeros((L, n_pages, H, page, d), dtype=np.uint8) for _ in range(2)]
        self.scales = [np.zeros((L, n_pages, H)) for _ in range(2)]

    def write(self, kv, x, page_table, seq_off, seq_pos, l_begin=0):
        """Quantise x [n_layers][H][T][d]; values that are not finite are stored as 0."""
        val = e4m3_values()
        x = np.where(np.isfinite(x), np.asarray(x, dtype=np.float64), 0.0)
        codes, scales, page = self.codes[kv], self.scales[kv], self.page
        for s in range(len(seq_pos)):
            n, p = int(seq_off[s + 1] - seq_off[s]), int(seq_pos[s])
            at = p
            while at < p + n:
                pid, s0 = int(page_table[s][at // page]), at % page
                m = min(page - s0, p + n - at)
                t = int(seq_off[s]) + at - p
                for l in range(x.shape[0]):
                    for h in range(x.shape[1]):
                        new = x[l, h, t:t + m]
                        e = block_exponent(np.abs(new).max())
                        c = codes[l_begin + l, pid, h]
                        if s0:
                            was = int(np.log2(scales[l_begin + l, pid, h]))
                            e = max(e, was)
                            if e > was:
                                c[:s0] = e4m3_encode(val[c[:s0]] * 2.0 ** (was - e))
                        c[s0:s0 + m] = e4m3_encode(new * 2.0 ** -e)
                        scales[l_begin + l, pid, h] = 2.0 ** e
                at += m

    def sequence(self, kv, page_row, n, l, h):
        """The first n positions of a sequence, [n][d]."""
        ids = np.asarray(page_row[:-(-n // self.page)], dtype=np.int64)
        if n == 0:
            return np.zeros((0, self.codes[kv].shape[4]))
        x = e4m3_values()[self.codes[kv][l, ids, h]] * self.scales[kv][l, ids, h][:, None, None]
        return x.reshape(-1, x.shape[-1])[:n]

    def read(self, kv, page_table, seq_off, seq_pos, l_begin=0, n_layers=None):
        L, _, H, _, d = self.codes[kv].shape
        n_layers = L - l_begin if n_layers is None else n_layers
        out = np.zeros((n_layers, H, int(seq_off[-1]), d))
        for s in range(len(seq_pos)):
            a, b, p = int(seq_off[s]), int(seq_off[s + 1]), int(seq_pos[s])
            for l in range(n_layers):
                for h in range(H):
                    out[l, h, a:b] = self.sequence(kv, page_table[s], p + b - a, l_begin + l, h)[p:]
        return out

    def attention(self, q, page_table, seq_off, seq_pos, kv_len=None, l_begin=0, scale=None):
        """(out [n_layers][Hq][T][d], lse [n_layers][Hq][T], spread, reach).

        spread [n_layers][Hq][T][d] is sum_j p_j |v_j| and reach [n_layers][Hq][T] the
        largest scale * sum_e |q_e k_je| over visible j: what rounding errors scale with.
        """
        q = np.asarray(q, dtype=np.float64)
        n_layers, Hq, T, d = q.shape
        H = self.codes[0].shape[2]
        g = Hq // H
        scale = 1 / np.sqrt(d) if scale is None else scale
        out, spread = np.zeros(q.shape), np.zeros(q.shape)
        lse, reach = np.full(q.shape[:3], -np.inf), np.zeros(q.shape[:3])
        for s in range(len(seq_pos)):
            a, b, p = int(seq_off[s]), int(seq_off[s + 1]), int(seq_pos[s])
            kv = max(0, p + b - a if kv_len is None else int(kv_len[s]))
            if b == a or kv == 0:
                continue
            see = np.arange(kv)[None] <= p + np.arange(b - a)[:, None]
            for l in range(n_layers):
                for h in range(H):
                    k, v = (self.sequence(x, page_table[s], kv, l_begin + l, h) for x in (0, 1))
                    for hq in range(h * g, (h + 1) * g):
                        sc = np.where(see, scale * (q[l, hq, a:b] @ k.T), -np.inf)
                        m = sc.max(axis=1)
                        ok = m > -np.inf
                        w = np.exp(sc - np.where(ok, m, 0.0)[:, None])
                        tot = w.sum(axis=1)
                        w = w / np.where(ok, tot, 1.0)[:, None]
                        out[l, hq, a:b], spread[l, hq, a:b] = w @ v, w @ np.abs(v)
                        lse[l, hq, a:b] = np.where(ok, m + np.log(np.where(ok, tot, 1.0)), -np.inf)
                        r = scale * (np.abs(q[l, hq, a:b]) @ np.abs(k).T)
                        reach[l, hq, a:b] = np.where(see, r, 0.0).max(axis=1)
        return out, lse, spread, reach
