"""Plain counterparts of the paged-cache calls for the tests: sequential
Python over numpy tables for the page calls, float64 for the attention."""
from __future__ import annotations

import numpy as np

D = 128


def unit_list(n_seq, n_layers, n_kvheads, layer=-1):
    layers = range(n_layers) if layer < 0 else [layer]
    return [(s * n_layers + l) * n_kvheads + h for s in range(n_seq) for l in layers
            for h in range(n_kvheads)]


def attention(q, k, v, scale, dims=None):
    """q [G, D], k / v [n, D] float64 -> out [G, D], lse [G], and the error
    bound of a float32 evaluation of each output.  (``dims``: v holds these
    dims only.)

    The bound: a score is a sum of 128 products, each rounding of it at most
    2^-24 of the partial sum, at most A = scale sum |q_d k_d|; roundings of a
    sum of 128 terms add up as a random walk, sqrt(128) of them, taken 4 times
    (four standard deviations) for the products, the scale and the logarithm's
    base.  A weight is off by the score's and its maximum's error, 2 dS, and by
    exp2's 2^-22; the sums over the rows add 2^-24 a rounding, again as a
    random walk, taken 4 times.  The denominator is off by as much again."""
    G = q.shape[0]
    width = D if dims is None else len(dims)
    out, lse = np.zeros((G, width)), np.full(G, -np.inf)
    tol_o, tol_l = np.zeros((G, width)), np.zeros(G)
    n = len(k)
    if n == 0:
        return out, lse, tol_o, tol_l
    for h in range(G):
        s = (k @ q[h]) * scale
        m = s.max()
        p = np.exp(s - m)
        den = p.sum()
        out[h] = p @ v / den
        lse[h] = m + np.log(den)
        A = (np.abs(k) @ np.abs(q[h])).max() * scale
        eps = 2.0 ** -24
        ds = 4 * np.sqrt(D + 4) * eps * max(A, 1.0)
        rel = 2 * (2 * ds + 4 * eps + 4 * np.sqrt(n + 16) * eps)
        tol_o[h] = rel * (p @ np.abs(v) / den) + 1e-30
        tol_l[h] = rel + 4 * eps * abs(lse[h])
    return out, lse, tol_o, tol_l


class Pages:
    """A paged cache's tables as numpy arrays, changed one step after another."""

    def __init__(self, table, refs, n_valid, n_seq, rows):
        self.table, self.refs, self.n_valid = table.copy(), refs.copy(), n_valid.copy()
        self.n_seq, self.rows = n_seq, rows
        self.per_seq = table.shape[0] // n_seq
        self.copied = []  # (from page, to page, rows)

    def fit(self, n_add, own=False):
        U, ppu = self.table.shape
        for u in range(U):
            keep = -(-(int(self.n_valid[u]) + n_add[u // self.per_seq]) // self.rows)
            for s in range(keep, ppu):
                if self.table[u, s] >= 0:
                    self.refs[self.table[u, s]] -= 1
                    self.table[u, s] = -1
        holders = {}  # of shared pages that will be written, in (unit, slot) order
        want = []
        for u in range(U):
            n, add = int(self.n_valid[u]), n_add[u // self.per_seq]
            for s in range(-(-(n + add) // self.rows)):
                p = int(self.table[u, s])
                if p < 0:
                    want.append((u, s, -1))
                elif self.refs[p] > 1 and (own or (add > 0 and (s + 1) * self.rows > n)):
                    holders.setdefault(p, []).append((u, s))
                    want.append((u, s, p))
        keeps = {h[-1] for p, h in holders.items() if len(h) == self.refs[p]}
        want = [w for w in want if (w[0], w[1]) not in keeps]
        free = [p for p in range(len(self.refs)) if self.refs[p] == 0]
        n_free = len(free) - len(want)
        if n_free < 0:
            return n_free
        for (u, s, old), p in zip(want, free):
            if old >= 0:
                self.refs[old] -= 1
                r = min(self.rows, max(0, int(self.n_valid[u]) - s * self.rows))
                self.copied.append((old, p, r))
            self.refs[p] = 1
            self.table[u, s] = p
        return n_free

    def fork(self, src, dst, pos=None, p_cur=None):
        t0, n0 = self.table.copy(), self.n_valid.copy()
        x0 = None if pos is None else pos.copy()
        c0 = None if p_cur is None else p_cur.copy()
        taken, skipped = set(), 0
        for a, b in zip(src, dst):
            if not (-1 <= a < self.n_seq and 0 <= b < self.n_seq) or b in taken:
                skipped += 1
                taken.add(b)
                continue
            taken.add(b)
            for i in range(self.per_seq):
                ub, ua = b * self.per_seq + i, a * self.per_seq + i
                n = int(n0[ua]) if a >= 0 else 0
                for s in range(self.table.shape[1]):
                    if self.table[ub, s] >= 0:
                        self.refs[self.table[ub, s]] -= 1
                    p = t0[ua, s] if s * self.rows < n else -1
                    self.table[ub, s] = p
                    if p >= 0:
                        self.refs[p] += 1
                self.n_valid[ub] = n
                if pos is not None and a >= 0:
                    pos[ub, :n] = x0[ua, :n]
            if p_cur is not None:
                p_cur[b] = c0[a] if a >= 0 else 0
        return skipped

    def compact(self):
        live = int((self.refs != 0).sum())
        src = [p for p in range(live, len(self.refs)) if self.refs[p] != 0]
        dst = [p for p in range(live) if self.refs[p] == 0]
        to = dict(zip(src, dst))
        for a, b in to.items():
            self.copied.append((a, b, self.rows))
            self.refs[b], self.refs[a] = self.refs[a], 0
        for u in range(self.table.shape[0]):
            for s in range(self.table.shape[1]):
                p = int(self.table[u, s])
                self.table[u, s] = to.get(p, p)
        return live

    def check(self):
        """Every count is the number of entries that name the page."""
        named = np.bincount(self.table[self.table >= 0].ravel(), minlength=len(self.refs))
        assert np.array_equal(named, self.refs)
