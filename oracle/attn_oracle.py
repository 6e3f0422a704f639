"""CPU oracle of the attention operators and of the paged key-value cache.

TEST INFRASTRUCTURE ONLY, like staple_oracle: plain float64 numpy with loops,
sharing no code with the library.

A sequence's query i stands at position p = i + Lk - Lq and sees key j when
j <= p and (window == 0 or j > p - window or j < sinks).  Only visible pairs
enter any sum: a hidden key's rows are never multiplied, not even by zero.
"""
from __future__ import annotations

import numpy as np


def visible(lq: int, lk: int, window: int, sinks: int) -> np.ndarray:
    see = np.zeros((lq, lk), dtype=bool)
    for i in range(lq):
        p = i + lk - lq
        for j in range(min(p, lk - 1) + 1):
            see[i, j] = window == 0 or j > p - window or j < sinks
    return see


def _masked_product(w, x):
    """w @ x over w's non-zero entries alone (w [a, b], x [b, d])."""
    hidden = w == 0
    if np.all(np.isfinite(x)):
        return w @ x
    out = np.zeros((w.shape[0], x.shape[1]))
    for i in range(w.shape[0]):
        out[i] = w[i, ~hidden[i]] @ x[~hidden[i]]
    return out


def attend(q, k, v, see, scale, do=None):
    """One head of one sequence: o, lse, p, and with `do` dq, dk, dv, ds."""
    q, k, v = (np.asarray(a, dtype=np.float64) for a in (q, k, v))
    with np.errstate(invalid="ignore", over="ignore"):
        s = np.where(see, scale * (q @ k.T), -np.inf)
    empty = ~see.any(axis=1) if see.size else np.ones(len(q), dtype=bool)
    top = np.where(empty, 0.0, s.max(axis=1, initial=-np.inf))
    e = np.where(see, np.exp(s - top[:, None]), 0.0)
    total = e.sum(axis=1)
    p = e / np.where(empty, 1.0, total)[:, None]
    with np.errstate(divide="ignore"):
        out = {"p": p, "o": _masked_product(p, v), "lse": np.where(empty, -np.inf, top + np.log(total))}
    if do is not None:
        do = np.asarray(do, dtype=np.float64)
        with np.errstate(invalid="ignore"):
            dp = np.where(see, do @ v.T, 0.0)
            delta = (p * dp).sum(axis=1)
            ds = np.where(see, p * (dp - delta[:, None]), 0.0)
        out.update(ds=ds, dq=scale * _masked_product(ds, k), dk=scale * _masked_product(ds.T, q),
                   dv=_masked_product(p.T, do))
    return out


class Pages:
    """The cache's bookkeeping and contents, one step at a time."""

    def __init__(self, refs, table, lens, k, v):
        self.refs, self.table, self.lens = (np.array(a, dtype=np.int64) for a in (refs, table, lens))
        self.k, self.v = np.array(k), np.array(v)   # [layers, pages, heads, page, dim]
        self.page = self.k.shape[3]

    def held(self, s):
        return -(-int(self.lens[s]) // self.page)

    def free(self, seqs):
        for s in seqs:
            for j in range(self.held(s)):
                self.refs[self.table[s, j]] -= 1
                self.table[s, j] = -1
            self.lens[s] = 0

    def fork(self, parents, children):
        for a, c in zip(parents, children):
            assert self.lens[c] == 0
            for j in range(self.held(a)):
                self.table[c, j] = self.table[a, j]
                self.refs[self.table[a, j]] += 1
            self.lens[c] = self.lens[a]

    def extend(self, seqs, n_new):
        """False, with nothing changed, where pages or columns run out."""
        before = self.refs.copy()
        todo, need = [], 0
        for s, n in zip(seqs, n_new):
            old = int(self.lens[s])
            cow = n > 0 and old % self.page != 0 and before[self.table[s, self.held(s) - 1]] > 1
            more = -(-(old + n) // self.page) - self.held(s)
            if self.held(s) + more > self.table.shape[1]:
                return False
            todo.append((s, n, old, cow, more))
            need += more + cow
        free = [p for p in range(len(before)) if before[p] == 0]
        if need > len(free):
            return False
        for s, n, old, cow, more in todo:
            col = self.held(s)
            if cow:
                a, b = self.table[s, col - 1], free.pop(0)
                used = old % self.page
                self.k[:, b, :, :used] = self.k[:, a, :, :used]
                self.v[:, b, :, :used] = self.v[:, a, :, :used]
                self.refs[a] -= 1
                self.refs[b] = 1
                self.table[s, col - 1] = b
            for j in range(more):
                b = free.pop(0)
                self.refs[b] = 1
                self.table[s, col + j] = b
            self.lens[s] = old + n
        return True

    def append(self, seqs, rows_k, rows_v, layer=0):
        """rows_k[i], rows_v[i]: the last tokens of seqs[i], [n, heads, dim]."""
        for s, a, b in zip(seqs, rows_k, rows_v):
            for t in range(len(a)):
                pos = int(self.lens[s]) - len(a) + t
                p = self.table[s, pos // self.page]
                self.k[layer, p, :, pos % self.page] = a[t]
                self.v[layer, p, :, pos % self.page] = b[t]

    def rows(self, pool, s, layer=0):
        """The cached rows of a sequence, [len, heads, dim]."""
        return np.array([pool[layer, self.table[s, j // self.page], :, j % self.page]
                         for j in range(int(self.lens[s]))]).reshape(-1, pool.shape[2], pool.shape[4])

    def compact(self):
        live = [p for p in range(len(self.refs)) if self.refs[p] > 0]
        n = len(live)
        movers = [p for p in live if p >= n]
        holes = [p for p in range(n) if self.refs[p] <= 0]
        to = dict(zip(movers, holes))
        for a, b in to.items():
            self.k[:, b], self.v[:, b] = self.k[:, a], self.v[:, a]
            self.refs[b], self.refs[a] = self.refs[a], 0
        for s in range(len(self.lens)):
            for j in range(self.held(s)):
                self.table[s, j] = to.get(int(self.table[s, j]), self.table[s, j])
        return n
