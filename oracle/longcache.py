"""fp64 CPU oracle of the calls for long caches -- TEST INFRASTRUCTURE.

Plain numpy and Python lists, written from the definitions in ``dsel.h``: the 4-bit
format value by value, what a query sees under a sliding window one key at a time,
the accumulated weight of a position, and the positions that eviction keeps.
"""
from __future__ import annotations

import numpy as np

from .tree import Pool

MXFP4 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def to_mxfp4(x):
    """Codes (one an element) and scale bytes of values ``[..., n]``, n a multiple of
    32.  The exponent is found by trying, the code by the distance to each value."""
    x = np.asarray(x, np.float64)
    b = x.reshape(*x.shape[:-1], x.shape[-1] // 32, 32)
    top = np.abs(b).max(-1)
    fine = np.isfinite(top)
    e = np.full(top.shape, 125)
    for k in range(125, -124, -1):
        e = np.where(top <= 7 * 2.0 ** k, k, e)
    y = np.where(fine[..., None], np.abs(b) / 2.0 ** e[..., None], 0.0)
    order = [0, 2, 4, 6, 1, 3, 5, 7]  # of two as near, the even code
    gap = np.abs(y[..., None] - MXFP4[order])
    code = np.array(order)[gap.argmin(-1)] + 8 * np.signbit(b)
    code = np.where(fine[..., None], code, 0)
    return code.reshape(x.shape).astype(np.uint8), np.where(fine, e + 127, 255).astype(np.uint8)


def from_mxfp4(code, byte):
    """The values of codes ``[..., n]`` under scale bytes ``[..., n / 32]`` (255: NaN)."""
    v = MXFP4[code & 7] * np.where(code & 8, -1.0, 1.0)
    s = np.where(byte == 255, np.nan, 2.0 ** (byte.astype(np.float64) - 127))
    return v * np.repeat(s, 32, -1)


def pack(code):
    """Two codes a byte, the first in the low bits."""
    return code[..., 0::2] | (code[..., 1::2] << 4)


def unpack(byte):
    return np.stack([byte & 15, byte >> 4], -1).reshape(*byte.shape[:-1], -1)


def window_sees(sees, s, depth, window, sinks):
    """Truth values ``[n, s + n]`` narrowed to what lies in a window or among the sinks;
    ``depth [n]``."""
    out = sees.copy()
    at = list(range(s)) + [s + int(d) for d in depth]
    for i in range(sees.shape[0]):
        for j in range(sees.shape[1]):
            if not (at[j] < sinks or s + int(depth[i]) - at[j] < window):
                out[i, j] = False
    return out


def key_weights(q, lse, K, scale, count=None):
    """Sums ``[N]`` over the queries of ``count e^(z - lse)``: ``q [n, Hq, D]``, ``lse [n,
    Hq]``, ``K [N, H, D]``; a query whose lse is not finite counts nothing.  Also the
    sums of ``count e^(z - lse) zmag``, for error bounds, zmag being sum |q||K| scale."""
    n, Hq, D = q.shape
    g = Hq // K.shape[1]
    out, mag = np.zeros(len(K)), np.zeros(len(K))
    for i in range(n):
        for h in range(Hq):
            if not np.isfinite(lse[i, h]) or (count is not None and not count[i] > 0):
                continue
            p = np.exp(K[:, h // g] @ q[i, h] * scale - lse[i, h]) * (1.0 if count is None else count[i])
            out += p
            mag += p * (np.abs(K[:, h // g]) @ np.abs(q[i, h]) * abs(scale))
    return out, mag


def keep(weights, n, budget, sinks, recent):
    """The positions of ``n`` that stay, ascending: the sinks, the last ones, then by
    weight (NaN below all, the lowest position of equals)."""
    fixed = [p for p in range(n) if p < sinks or p >= n - recent]
    rest = [p for p in range(n) if sinks <= p < n - recent]
    rest.sort(key=lambda p: (-np.inf if np.isnan(weights[p]) else weights[p], not np.isnan(weights[p]), -p), reverse=True)
    return sorted(fixed + rest[:budget - len(fixed)])


class LongPool(Pool):
    """The pool with eviction, one row at a time."""

    def evict(self, budget, weights, sinks, recent):
        """(granted, kept): ``weights [rows, ld]`` is changed in place; kept[r] is a list, or None where
        the row stays as it is."""
        cut = [r for r in range(len(budget)) if 0 <= budget[r] < self.seq_len[r] and budget[r] >= sinks + recent]
        need = {r: -(-int(budget[r]) // self.P) for r in cut}
        pages = self._take(sum(need.values()))
        kept = [None] * len(budget)
        if pages is None:
            return 0, kept
        old = []
        for r in cut:
            n, K = int(self.seq_len[r]), int(budget[r])
            kept[r] = keep(weights[r], n, K, sinks, recent)
            fresh = [pages.pop(0) for _ in range(need[r])]
            for c in self.caches:
                for i, p in enumerate(kept[r]):
                    c[:, fresh[i // self.P], i % self.P] = c[:, self.table[r, p // self.P], p % self.P]
            old += [(r, int(p)) for p in self.table[r, :self.row_pages[r]]]
            w = weights[r, kept[r]].copy()
            weights[r, :n] = 0
            weights[r, :K] = w
            self.table[r, :self.row_pages[r]] = -1
            self.table[r, :need[r]] = fresh
            self.row_pages[r], self.seq_len[r] = need[r], K
            self.refcount[fresh] = 1
        for _, p in old:
            self.refcount[p] -= 1
        return 1, kept
