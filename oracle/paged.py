"""Plain reference of the paged cache and its attention: one sequence, one
page, one row at a time, attention in fp64.

The pages of the method name no paged cache; the rules are those include/tv.h
states at tv_pool, tv_pages_* and tv_attend_*.  Pool values are kept as the
uint16 bit patterns of bf16.
"""
from __future__ import annotations

import numpy as np


class Refused(Exception):
    """The call's status; nothing has changed."""


class Cache:
    """A pool and its sequence table, as the calls see them."""

    def __init__(self, k, v, refs, pages, lens):
        self.k, self.v = k, v              # [layers][pages][heads][page_size][dim] uint16
        self.refs, self.pages, self.lens = refs, pages, lens

    @property
    def ps(self):
        return self.k.shape[3]

    def _held(self, n):
        return -(-n // self.ps)

    def _len(self, s):
        if not 0 <= s < len(self.lens) or not 0 <= self.lens[s] <= self.pages.shape[1] * self.ps:
            raise Refused("TV_E_SEQ")
        return int(self.lens[s])

    def _page(self, s, j):
        p = int(self.pages[s, j])
        if not 0 <= p < len(self.refs) or self.refs[p] < 1:
            raise Refused("TV_E_PAGE")
        return p

    def _once(self, ids):
        if len(set(ids)) < len(ids):
            raise Refused("TV_E_SEQ")

    def extend(self, ids, add):
        self._once(ids)
        for s, a in zip(ids, add):
            n = self._len(s)
            if a < 0:
                raise Refused("TV_E_SEQ")
            if n + a > self.pages.shape[1] * self.ps:
                raise Refused("TV_E_CAPACITY")
            if a and n % self.ps:
                self._page(s, n // self.ps)
        refs, todo = self.refs.copy(), []
        free = [p for p in range(len(refs)) if refs[p] == 0]
        for s, a in zip(ids, add):
            n = int(self.lens[s])
            have = self._held(n)
            if a and n % self.ps and refs[self.pages[s, have - 1]] > 1:
                refs[self.pages[s, have - 1]] -= 1
                todo.append((s, have - 1, int(self.pages[s, have - 1])))
            todo += [(s, j, None) for j in range(have, self._held(n + a))]
        if len(todo) > len(free):
            raise Refused("TV_E_CAPACITY")
        self.refs[:] = refs
        for (s, j, old), p in zip(todo, free):
            self.refs[p] = 1
            self.pages[s, j] = p
            if old is not None:
                self.k[:, p], self.v[:, p] = self.k[:, old], self.v[:, old]
        for s, a in zip(ids, add):
            self.lens[s] += a

    def fork(self, src, dst):
        self._once(dst)
        for s, d in zip(src, dst):
            if not 0 <= d < len(self.lens) or self.lens[d] != 0 or d in src:
                raise Refused("TV_E_SEQ")
            for j in range(self._held(self._len(s))):
                self._page(s, j)
        for s, d in zip(src, dst):
            for j in range(self._held(int(self.lens[s]))):
                self.pages[d, j] = self.pages[s, j]
                self.refs[self.pages[s, j]] += 1
            self.lens[d] = self.lens[s]

    def release(self, ids, keep):
        self._once(ids)
        for s, m in zip(ids, keep):
            n = self._len(s)
            if not 0 <= m <= n:
                raise Refused("TV_E_SEQ")
            for j in range(self._held(m), self._held(n)):
                self._page(s, j)
        for s, m in zip(ids, keep):
            for j in range(self._held(m), self._held(int(self.lens[s]))):
                self.refs[self.pages[s, j]] -= 1
            self.lens[s] = m

    def compact(self):
        for s in range(len(self.lens)):
            for j in range(self._held(self._len(s))):
                self._page(s, j)
        used = int((self.refs > 0).sum())
        src = [p for p in range(used, len(self.refs)) if self.refs[p] > 0]
        dst = [p for p in range(used) if self.refs[p] == 0]
        remap = np.where(self.refs > 0, np.arange(len(self.refs)), -1).astype(np.int32)
        for a, b in zip(src, dst):
            remap[a] = b
            self.k[:, b], self.v[:, b] = self.k[:, a], self.v[:, a]
            self.refs[b], self.refs[a] = self.refs[a], 0
        for s in range(len(self.lens)):
            for j in range(self._held(int(self.lens[s]))):
                self.pages[s, j] = remap[self.pages[s, j]]
        return remap, used

    def slot(self, s, t):
        return int(self.pages[s, t // self.ps]), t % self.ps

    def write(self, layer, s, pos, k, v):
        """k, v [rows][heads][dim] into tokens pos, pos + 1, ... of sequence s."""
        if pos < 0 or pos + len(k) > self._len(s):
            raise Refused("TV_E_CAPACITY")
        for r in range(len(k)):
            p, o = self.slot(s, pos + r)
            self.k[layer, p, :, o], self.v[layer, p, :, o] = k[r], v[r]

    def rows(self, layer, s, pos, n):
        """The other way: (k, v) [n][heads][dim]."""
        at = [self.slot(s, pos + r) for r in range(n)]
        shape = (n, self.k.shape[2], self.k.shape[4])
        return tuple(np.array([x[layer, p, :, o] for p, o in at], dtype=np.uint16).reshape(shape) for x in (self.k, self.v))


def attend(q, k, v, spread=False):
    """softmax(q k^T / sqrt(D)) v in fp64: q [heads][D], k and v [tokens][kv_heads][D]; no token gives zeros.
    With spread also sum_j w_j |v_j - o| (weights w), what a relative error of every weight can move the result by."""
    heads, dim = q.shape
    out, off = np.zeros((heads, dim)), np.zeros((heads, dim))
    group = heads // k.shape[1]
    for h in range(heads if len(k) else 0):
        a = k[:, h // group] @ q[h] / np.sqrt(dim)
        p = np.exp(a - a.max())
        p /= p.sum()
        out[h] = p @ v[:, h // group]
        if spread:
            off[h] = p @ np.abs(v[:, h // group] - out[h])
    return (out, off) if spread else out


def attend_prompt(q, k, v, starts, spread=False):
    """Causal attention of packed sequences: row t of a sequence sees its rows 0..t.  q [rows][heads][D]; rows outside
    every sequence are NaN here (the call leaves them as they were)."""
    out, off = np.full(q.shape, np.nan), np.zeros(q.shape)
    for a, b in zip(starts[:-1], starts[1:]):
        for t in range(a, b):
            out[t], off[t] = attend(q[t], k[a:t + 1], v[a:t + 1], True)
    return (out, off) if spread else out
