"""Paged KV cache: rotary positions, attention over pages, row compaction, page lifecycle (oracle, test infrastructure).

Graft article, architecture paragraph: the merged tree is verified in one
target forward over the prefix cache, and the accepted nodes' rows join it.
Here the cache lies in pages (pool [P][R][H][d], a row of page numbers a
sequence); everything is written out in float64 from the definitions:

    rotary      (x, y) -> f (x cos a - y sin a, x sin a + y cos a),  a = position * w
    attention   o = sum_j softmax_j(scale q . k_j) v_j over the rows a new row sees
    compaction  row L + t <- row L + path[t]
    pages       reference counts; the lowest free pages first; copy on write
"""
from __future__ import annotations

import numpy as np


def rope(x: np.ndarray, pos, inv_freq, interleaved: bool, factor: float) -> np.ndarray:
    """x [N][H][d]; turns the first 2 len(inv_freq) dims of every head."""
    x = x.astype(np.float64)
    out = x.copy()
    half = len(inv_freq)
    a = np.asarray(pos, np.float64)[:, None, None] * np.asarray(inv_freq, np.float64)
    c, s = factor * np.cos(a), factor * np.sin(a)
    i = np.arange(half)
    p, q = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    out[..., p] = x[..., p] * c - x[..., q] * s
    out[..., q] = x[..., p] * s + x[..., q] * c
    return out


def rows(pool: np.ndarray, table_row, n: int) -> np.ndarray:
    """The first n rows of a sequence, [n][H][d]."""
    R = pool.shape[1]
    return np.stack([pool[table_row[r // R], r % R] for r in range(n)]) if n else pool[0, :0]


def attention(Q, K, V, table, lengths, q_start, scale: float, mask=None, absolute: bool = False):
    """Q [N][Hq][d], K, V pools.  Returns float64 [N][Hq][d], NaN in rows outside every sequence; with
    ``absolute``, also the same weights applied to |V| (the scale of the sums, for error bounds)."""
    N, Hq, d = Q.shape
    group = Hq // K.shape[2]
    out = np.full((N, Hq, d), np.nan)
    size = np.full((N, Hq, d), np.nan)
    for b in range(len(lengths)):
        lo, hi, L = int(q_start[b]), int(q_start[b + 1]), int(lengths[b])
        if hi == lo:
            continue
        k = rows(K, table[b], L + hi - lo).astype(np.float64)
        v = rows(V, table[b], L + hi - lo).astype(np.float64)
        n = hi - lo
        seen = np.ones((n, L + n), bool)
        for i in range(n):
            if mask is None:
                seen[i] = np.arange(L + n) <= L + i
            else:
                bits = int(mask[lo + i]) & (2**64 - 1)
                seen[i, L:] = [bool(bits >> j & 1) for j in range(n)]
        some = seen.any(1)
        for h in range(Hq):
            # (what a row does not see takes no part: its products may be NaN)
            with np.errstate(invalid="ignore"):
                s = np.where(seen, Q[lo:hi, h].astype(np.float64) @ k[:, h // group].T * scale, -np.inf)
            w = np.exp(s - np.where(some, s.max(1), 0.0)[:, None])
            w /= np.where(some, w.sum(1), 1.0)[:, None]
            vh = v[:, h // group]
            odd = ~np.isfinite(vh)
            out[lo:hi, h] = w @ np.where(odd, 0.0, vh)
            size[lo:hi, h] = w @ np.abs(np.where(odd, 0.0, vh))
            for j, c in zip(*np.nonzero(odd)):
                out[lo:hi, h, c] += np.where(seen[:, j], vh[j, c], 0.0)
    return (out, size) if absolute else out


def compact(K, V, table, lengths, path, acc_len):
    """K, V [layers][P][R][H][d]; returns new arrays and lengths."""
    K, V, R = K.copy(), V.copy(), K.shape[2]
    for b in range(len(lengths)):
        for t in range(int(acc_len[b])):
            x, y = int(lengths[b]) + int(path[b][t]), int(lengths[b]) + t
            for pool in (K, V):
                pool[:, table[b][y // R], y % R] = pool[:, table[b][x // R], x % R]
    return K, V, np.asarray(lengths) + np.asarray(acc_len)


class Pages:
    """Block table, held counts, lengths and reference counts, one operation at a time."""

    def __init__(self, table, held, lengths, refs, R: int):
        self.table = [list(map(int, r)) for r in table]
        self.held, self.lengths, self.refs = list(map(int, held)), list(map(int, lengths)), list(map(int, refs))
        self.R = R

    def free(self, seqs):
        for b in dict.fromkeys(int(x) for x in seqs):
            for p in self.table[b][:self.held[b]]:
                self.refs[p] -= 1
            self.table[b] = [-1] * len(self.table[b])
            self.held[b] = self.lengths[b] = 0

    def fork(self, src, dst):
        for a, b in zip(src, dst):
            n = -(-self.lengths[a] // self.R)
            self.table[b] = self.table[a][:n] + [-1] * (len(self.table[b]) - n)
            for p in self.table[b][:n]:
                self.refs[p] += 1
            self.held[b], self.lengths[b] = n, self.lengths[a]

    def reserve(self, new_rows):
        """Returns (copies, refused): copies are (old page, new page, rows below the length)."""
        before = list(self.refs)
        fresh = [p for p, r in enumerate(before) if r == 0]
        copies, refused, taken = [], [], 0
        for b, n in enumerate(new_rows):
            if n <= 0:
                continue
            L = self.lengths[b]
            last = -(-(L + n) // self.R)
            wanted = [j for j in range(L // self.R, last)
                      if j >= self.held[b] or before[self.table[b][j]] > 1]
            if wanted and taken + len(wanted) > len(fresh):
                refused.append(b)
                taken += len(wanted)
                continue
            for j in wanted:
                new, taken = fresh[taken], taken + 1
                old = self.table[b][j] if j < self.held[b] else -1
                if old >= 0:
                    self.refs[old] -= 1
                    if L > j * self.R:
                        copies.append((old, new, L - j * self.R))
                self.refs[new] = 1
                self.table[b][j] = new
            self.held[b] = max(self.held[b], last)
        return copies, refused
