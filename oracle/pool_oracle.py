"""Slow definitions of the shared pool's calls (share, reserve, truncate, compact) on
numpy copies of a cache's tables, and of the verification of drafted tokens in 64
bits.  numpy only; written from include/shadowkv.h, independent of the library's code."""
from __future__ import annotations

import numpy as np


class Pool:
    """table (b, h, max_blocks), n_tok (b, h), weight, refs (n_pool,); content[id]: whatever a block holds."""

    def __init__(self, table, n_tok, weight, refs, block, content):
        self.table, self.n_tok, self.weight, self.refs = (np.array(x) for x in (table, n_tok, weight, refs))
        self.block, self.content = block, list(content)

    def blocks(self, n):
        return -(-int(n) // self.block)

    def share(self, src, dst):
        """The forks left out."""
        b, old, out = len(self.table), (self.table.copy(), self.n_tok.copy(), self.weight.copy()), []
        for k, (s, d) in enumerate(zip(src, dst)):
            if not (0 <= s < b and 0 <= d < b) or d in list(src) or d in list(dst)[:k]:
                out.append(k)
                continue
            for g in range(self.table.shape[1]):
                for i in range(self.table.shape[2]):
                    if self.table[d, g, i] >= 0:
                        self.refs[self.table[d, g, i]] -= 1
                    new = old[0][s, g, i] if i < self.blocks(old[1][s, g]) else -1
                    if new >= 0:
                        self.refs[new] += 1
                    self.table[d, g, i] = new
            self.n_tok[d], self.weight[d] = old[1][s], old[2][s]
        return out

    def truncate(self, drop=None):
        for i, g in np.ndindex(*self.n_tok.shape):
            n = self.n_tok[i, g] = max(0, int(self.n_tok[i, g]) - (0 if drop is None else max(0, int(drop[i]))))
            for e in range(self.blocks(n), self.table.shape[2]):
                if self.table[i, g, e] >= 0:
                    self.refs[self.table[i, g, e]] -= 1
                self.table[i, g, e], self.weight[i, g, e] = -1, 0

    def reserve(self, lens):
        b, h, mb = self.table.shape
        refs, table = self.refs.copy(), self.table.copy()          # as the call found them
        free = [i for i in range(len(refs)) if refs[i] == 0]
        granted, asked = np.zeros(b, np.int64), 0
        for i in range(b):
            want, ok = [], True
            for g in range(h):
                n = int(self.n_tok[i, g])
                ok &= n + lens[i] <= mb * self.block
                if n % self.block:
                    ok &= table[i, g, n // self.block] >= 0
                if ok:
                    for e in range(n // self.block, self.blocks(n + lens[i])):
                        if table[i, g, e] < 0 or refs[table[i, g, e]] != 1:
                            want.append((g, e, e == n // self.block and n % self.block > 0))
            if not ok:
                continue
            at, asked = asked, asked + len(want)
            if want and asked > len(free):
                continue
            granted[i] = lens[i]
            for (g, e, copied), new in zip(want, free[at:]):
                old = table[i, g, e]
                if old >= 0:
                    self.refs[old] -= 1
                    if copied:
                        self.content[new] = self.content[old]
                self.refs[new] = 1
                self.table[i, g, e] = new
        return granted

    def compact(self):
        """Ids of the blocks in use, in their new order."""
        return [i for i in range(len(self.refs)) if self.refs[i] > 0]


def verify(logits, drafts, probs, accept, sample, n, temperature):
    """(tokens accepted, next token, how near a decision was to its border) of one sequence:
    logits (n + 1, V), drafts (n,), probs (n, V) or None, accept (n,), in 64 bits.  The nearness is
    relative to the numbers compared."""
    near = np.inf
    for j in range(n + 1):
        x = np.array(logits[j], np.float64)
        x[np.isnan(x)] = -np.inf
        x = np.minimum(x, np.finfo(np.float32).max)
        if temperature > 0 and np.any(x > -np.inf):
            p = np.exp((x - x.max()) / temperature)
            p /= p.sum()
        else:
            p = np.zeros_like(x)
            if np.any(x > -np.inf):
                p[int(np.argmax(x))] = 1.0
        if j == n:
            break
        y = int(drafts[j])
        q = np.array(probs[j], np.float64) if probs is not None else None
        if not 0 <= y < len(p):
            break
        left, right = float(accept[j]) * (1.0 if q is None else q[y]), p[y]
        if left != right:
            near = min(near, abs(left - right) / max(abs(left), abs(right)))
        if left < right:
            continue
        break
    a = j
    rest = p
    if a < n:
        if probs is None:
            rest = p.copy()
            if 0 <= int(drafts[a]) < len(p):
                rest[int(drafts[a])] = 0.0
        else:
            rest = np.maximum(p - np.array(probs[a], np.float64), 0.0)
        if rest.sum() <= 0:
            rest = p
    if rest.sum() <= 0:
        return a, -1, near
    cum = np.cumsum(rest)
    at = float(sample) * cum[-1]
    t = int(np.searchsorted(cum, at, side="right"))
    near = min(near, np.abs(cum - at)[cum != at].min() / cum[-1])
    return a, t, near
