"""fp64 CPU oracle of the tree operators and the paged cache -- TEST INFRASTRUCTURE.

Plain numpy and Python lists, written from the definitions in ``dsel.h``: a node's
ancestors by climbing, attention one query at a time over the keys that it sees,
the pool one row and one page at a time.
"""
from __future__ import annotations

import numpy as np


def ancestors(parent):
    """Ancestor-or-self truth values ``[T, T]`` and depths ``[T]`` of one tree (a
    list of parents; a link that goes to no earlier node makes a root)."""
    T = len(parent)
    vis, depth = np.zeros((T, T), bool), np.zeros(T, np.int32)
    for i in range(T):
        p = int(parent[i])
        if i > 0 and 0 <= p < i:
            vis[i] = vis[p]
            depth[i] = depth[p] + 1
        vis[i, i] = True
    return vis, depth


def pack(vis):
    """``[..., T, T]`` truth values as int32 words, bit j % 32 of word j / 32."""
    T = vis.shape[-1]
    words = np.zeros(vis.shape[:-1] + ((T + 31) // 32,), np.uint32)
    for j in range(T):
        words[..., j // 32] |= vis[..., j].astype(np.uint32) << np.uint32(j % 32)
    return words.view(np.int32)


def accept(parent, tok, target):
    """(path, out_tok) of one tree: lists of the kept nodes and of the tokens."""
    path, out, cur = [], [], 0 if len(parent) else -1
    while cur >= 0:
        path.append(cur)
        out.append(int(target[cur]))
        cur = next((c for c in range(cur + 1, len(parent)) if parent[c] == cur and tok[c] == target[cur]), -1)
    return path, out


def attend(q, K, V, sees, scale):
    """One sequence: ``q [n, Hq, D]``, ``K, V [N, H, D]`` fp64, ``sees [n, N]``.
    Returns ``out [n, Hq, D]``, ``lse [n, Hq]``, and for error bounds ``mag``, the
    sum of weight times |V| per output, and ``zmag [n, Hq]``, the largest sum of
    |q||K| scale over the keys seen."""
    n, Hq, D = q.shape
    g = Hq // K.shape[1]
    out, mag = np.zeros((n, Hq, D)), np.zeros((n, Hq, D))
    lse, zmag = np.full((n, Hq), -np.inf), np.zeros((n, Hq))
    for i in range(n):
        idx = np.nonzero(sees[i])[0]
        if len(idx) == 0:
            continue
        for h in range(Hq):
            Kh, Vh = K[idx, h // g], V[idx, h // g]
            with np.errstate(invalid="ignore", over="ignore"):
                z = Kh @ q[i, h] * scale
                top = z.max()
                p = np.exp(z - top)
                lse[i, h] = top + np.log(p.sum())
                p = p / p.sum()
                out[i, h] = (p[:, None] * Vh).sum(0)
                mag[i, h] = (p[:, None] * np.abs(Vh)).sum(0)
                zmag[i, h] = (np.abs(Kh) @ np.abs(q[i, h])).max() * abs(scale)
    return out, lse, mag, zmag


_E4M3 = None


def e4m3_values():
    """The 256 values of the 8-bit format (code 0x7F and 0xFF are NaN)."""
    global _E4M3
    if _E4M3 is None:
        v = np.zeros(256)
        for c in range(256):
            e, m = (c >> 3) & 15, c & 7
            x = m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
            v[c] = np.nan if (c & 127) == 127 else (-x if c & 128 else x)
        _E4M3 = v
    return _E4M3


def to_e4m3(x):
    """Codes of the nearest 8-bit values (ties to an even code), held to +-448."""
    pos = e4m3_values()[:127]
    x = np.asarray(x, np.float64)
    a = np.minimum(np.abs(x), 448.0)
    hi = np.clip(np.searchsorted(pos, a, side="left"), 0, 126)
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - pos[lo], pos[hi] - a
    c = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi).astype(np.uint8)
    c = np.where(np.isnan(x), 127, c).astype(np.uint8)
    return c | (np.signbit(x).astype(np.uint8) << 7)


class Pool:
    """The pool of pages, one row and one page at a time; every cache is a list of
    arrays ``[layers, pages, page_size, ...]``."""

    def __init__(self, table, row_pages, seq_len, refcount, page_size, caches=()):
        self.table, self.row_pages, self.seq_len, self.refcount = (np.array(a) for a in
                                                                   (table, row_pages, seq_len, refcount))
        self.P, self.caches = page_size, [np.array(c) for c in caches]

    def _take(self, n):
        free = [p for p in range(len(self.refcount)) if self.refcount[p] == 0]
        return free[:n] if len(free) >= n else None

    def free(self, which):
        for r in np.nonzero(which)[0]:
            for i in range(self.row_pages[r]):
                self.refcount[self.table[r, i]] -= 1
                self.table[r, i] = -1
            self.row_pages[r] = self.seq_len[r] = 0

    def reserve(self, extra):
        need = [max(0, -(-(int(self.seq_len[r]) + int(extra[r])) // self.P) - int(self.row_pages[r]))
                for r in range(len(extra))]
        need = [0 if self.row_pages[r] + n > self.table.shape[1] else n for r, n in enumerate(need)]
        pages = self._take(sum(need))
        if pages is None:
            return 0
        for r, n in enumerate(need):
            for _ in range(n):
                page = pages.pop(0)
                self.table[r, self.row_pages[r]] = page
                self.row_pages[r] += 1
                self.refcount[page] = 1
        return 1

    def fork(self, src):
        want = [r for r in range(len(src)) if src[r] >= 0]
        pages = self._take(sum(1 for r in want if self.seq_len[src[r]] % self.P))
        if pages is None:
            return 0
        for r in want:
            s, n = src[r], int(self.seq_len[src[r]])
            whole, rest = divmod(n, self.P)
            for i in range(whole):
                self.table[r, i] = self.table[s, i]
                self.refcount[self.table[s, i]] += 1
            if rest:
                page = pages.pop(0)
                self.table[r, whole] = page
                self.refcount[page] = 1
                for c in self.caches:
                    c[:, page, :rest] = c[:, self.table[s, whole], :rest]
            self.row_pages[r] = whole + (rest > 0)
            self.seq_len[r] = n
        return 1
