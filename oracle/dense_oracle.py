"""Slow 64-bit definitions of the dense decode path: the norm and rotation of
query and key heads, the e4m3 block cache's quantisation, attention over it,
and its eviction by gathered weight.  numpy only; written from the formulas in
include/shadowkv.h, independent of the library's code."""
from __future__ import annotations

import math

import numpy as np

SCALE_MIN = 2.0 ** -100


def norm_rope(x, weight, eps, norm, theta, rot, pos):
    """x (b, h, s, d), pos (b, s): (y, mag), mag_i = the sum of the magnitudes y_i is made of."""
    x = np.asarray(x, np.float64)
    if norm:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
        if weight is not None:
            x = x * np.asarray(weight, np.float64)
    y, mag = x.copy(), np.abs(x)
    half = rot // 2
    if half:
        # angles in turns, reduced exactly: pos is an integer below 2^31 and the
        # frequency a long double
        f = np.array([np.longdouble(theta) ** (np.longdouble(-2 * i) / rot) for i in range(half)]) / (
            2 * np.longdouble(math.pi) + np.longdouble(2.4492935982947064e-16))
        turns = np.asarray(pos, np.longdouble)[:, None, :, None] * f
        ang = ((turns - np.floor(turns)).astype(np.float64)) * 2 * math.pi
        c, s = np.cos(ang), np.sin(ang)
        a, b = x[..., :half], x[..., half:rot]
        y[..., :half] = a * c - b * s
        y[..., half:rot] = b * c + a * s
        mag[..., :half] = mag[..., half:rot] = np.abs(a) + np.abs(b)
    return y, mag


def e4m3(v):
    """Round to the nearest e4m3 number (ties to even), saturating at 448."""
    v = np.asarray(v, np.float64)
    a = np.minimum(np.abs(v), 448.0)
    with np.errstate(divide="ignore", invalid="ignore"):
        e = np.where(a > 0, np.floor(np.log2(np.where(a > 0, a, 1.0))), -6)
    step = 2.0 ** (np.maximum(e, -6) - 3)
    return np.copysign(np.minimum(np.rint(a / step) * step, 448.0), v)   # rint: ties to even


def block_scale(x):
    """Smallest 2^e, e >= -100, with max |finite x| <= 448 2^e."""
    a = np.abs(np.asarray(x, np.float64))
    m = a[np.isfinite(a)].max(initial=0.0)
    e = -100
    while m > 448.0 * 2.0 ** e:
        e += 1
    return 2.0 ** e


class Cache:
    """Per pair a list of (values' codes (block, d), scale) for K and V."""

    def __init__(self, b, h, d, block, max_blocks):
        self.b, self.h, self.d, self.block, self.max_blocks = b, h, d, block, max_blocks
        self.blocks = {(i, g): [] for i in range(b) for g in range(h)}   # [kc, ks, vc, vs]
        self.n = {p: 0 for p in self.blocks}
        self.weight = {p: [] for p in self.blocks}

    def append(self, k, v, lens):
        B = self.block
        for (i, g), bl in self.blocks.items():
            at, left, t = self.n[i, g], int(lens[i]), 0
            left = min(left, self.max_blocks * B - at)
            while left > 0:
                r = at % B
                n = min(left, B - r)
                if r == 0:
                    bl.append([np.zeros((B, self.d)), 0.0, np.zeros((B, self.d)), 0.0])
                    self.weight[i, g].append(0.0)
                for x, c in ((k, 0), (v, 2)):
                    new = np.asarray(x[i, g, t:t + n], np.float64)
                    s = max(block_scale(new), abs(bl[-1][c + 1]))
                    if r:
                        bl[-1][c][:r] = e4m3(bl[-1][c][:r] * (bl[-1][c + 1] / s))
                    bl[-1][c][r:r + n] = e4m3(new / s)
                    bl[-1][c + 1] = s
                at, left, t = at + n, left - n, t + n
            self.n[i, g] = at

    def values(self, i, g):
        n, bl = self.n[i, g], self.blocks[i, g]
        cat = lambda c: np.concatenate([x[c] * x[c + 1] for x in bl])[:n] if bl else np.zeros((0, self.d))  # noqa: E731
        return cat(0), cat(2)

    def attend(self, q, scale, decay=None):
        """q (b, h_q, d): out, lse, mag (sum p |v|), logit magnitude (max sum |q k| scale) per
        head, and the sum over 128-token tiles of the tile's largest p times its largest 448 V scale."""
        b, hq, d = q.shape
        G = hq // self.h
        out, mag = np.zeros((b, hq, d)), np.zeros((b, hq, d))
        lse, lm, top = np.full((b, hq), -np.inf), np.zeros((b, hq)), np.zeros((b, hq))
        for i in range(b):
            for g in range(self.h):
                k, v = self.values(i, g)
                n = len(k)
                w = np.zeros(len(self.blocks[i, g]))
                for h in range(g * G, (g + 1) * G):
                    if not n:
                        continue
                    z = scale * (k @ q[i, h])
                    m = z.max()
                    p = np.exp(z - m)
                    lse[i, h] = m + math.log(p.sum())
                    p /= p.sum()
                    out[i, h], mag[i, h] = p @ v, p @ np.abs(v)
                    lm[i, h] = (abs(scale) * (np.abs(k) @ np.abs(q[i, h]))).max()
                    per = 128 // self.block
                    for t in range(0, n, 128):
                        vs = max(abs(x[3]) for x in self.blocks[i, g][t // self.block:t // self.block + per])
                        top[i, h] += p[t:t + 128].max() * 448 * vs
                    full = np.zeros(len(w) * self.block)
                    full[:n] = p
                    w += full.reshape(len(w), self.block).sum(1)
                if decay is not None:
                    self.weight[i, g] = list(decay * np.asarray(self.weight[i, g]) + w if decay else w)
        return out, lse, mag, lm, top


def evict(weight, n_tok, block, keep, sink, recent):
    """Old indices kept (ascending) and the tokens then held, for one pair."""
    n = -(-n_tok // block)
    if n <= keep:
        return list(range(n)), n_tok
    fixed = set(range(min(sink, n))) | set(range(max(0, n - recent), n))
    w = [(-math.inf if math.isnan(weight[j]) else weight[j], j) for j in range(n) if j not in fixed]
    # NaN below everything, also below -inf
    w.sort(key=lambda x: (math.isnan(weight[x[1]]), -x[0], x[1]))
    kept = sorted(fixed | {j for _, j in w[:keep - len(fixed)]})
    tail = n_tok - (n - 1) * block
    return kept, (len(kept) - 1) * block + tail if kept[-1] == n - 1 else len(kept) * block
