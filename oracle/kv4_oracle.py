"""fp64 CPU oracle of the 4-bit KV cache (recsa_kv4_*), written from the definition in
include/recsa.h.  One object is one (sequence, KV head); no code is shared with the
library or its binding."""
from __future__ import annotations

import numpy as np

GROUP = 32


def _bf16_spacing(x: np.ndarray) -> np.ndarray:
    """Distance of neighbouring bf16 numbers in the binade of x (8 significant bits)."""
    _, e = np.frexp(x)
    return np.ldexp(1.0, np.maximum(e - 8, -133))


def quantize(x: np.ndarray):
    """x [.., d] -> (codes, s, lo), the last two [.., d/32]; all fp64."""
    g = np.asarray(x, np.float64).reshape(*x.shape[:-1], x.shape[-1] // GROUP, GROUP)
    with np.errstate(all="ignore"):
        bad = ~np.isfinite(g).all(-1)
        g = np.where(bad[..., None], 0.0, g)
        least, most = g.min(-1), g.max(-1)
        sp = _bf16_spacing(least)
        lo = np.floor(least / sp) * sp
        s = (most - lo) / 15.0
        sp = _bf16_spacing(s)
        s = np.ceil(s / sp) * sp
        big = 2.0 ** 128
        bad |= (np.abs(lo) >= big) | (s >= big)
        t = (g - lo[..., None]) / np.where(s > 0, s, 1.0)[..., None]
        codes = np.where(s[..., None] > 0, np.minimum(np.rint(t), 15), 0.0)
    codes = np.where(bad[..., None], 0.0, codes)
    return codes, np.where(bad, 0.0, s), np.where(bad, np.nan, lo)


def value(x: np.ndarray) -> np.ndarray:
    codes, s, lo = quantize(x)
    return (lo[..., None] + s[..., None] * codes).reshape(x.shape)


class Unit:
    """The cache of one (sequence, KV head)."""

    def __init__(self, d: int, scale: float | None = None):
        self.k = np.zeros((0, d))
        self.v = np.zeros((0, d))
        self.pos = np.zeros(0, np.int64)
        self.w = np.zeros(0)
        self.seen = 0
        self.scale = d ** -0.5 if scale is None else scale

    def append(self, k, v):
        n = len(k)
        self.k = np.concatenate([self.k, value(np.asarray(k, np.float64))])
        self.v = np.concatenate([self.v, value(np.asarray(v, np.float64))])
        self.pos = np.concatenate([self.pos, np.arange(self.seen, self.seen + n)])
        self.w = np.concatenate([self.w, np.zeros(n)])
        self.seen += n

    def probabilities(self, q, at: int):
        """Softmax over the slots whose position is <= at (zeros elsewhere)."""
        p = np.zeros(len(self.k))
        sees = self.pos <= at
        if sees.any():
            s = self.k[sees] @ np.asarray(q, np.float64) * self.scale
            e = np.exp(s - s.max())
            p[sees] = e / e.sum()
        return p

    def attend(self, q, at: int, accumulate: bool = False):
        """q [G][d] at position `at`."""
        out = np.zeros((len(q), self.k.shape[1]))
        for i, x in enumerate(q):
            p = self.probabilities(x, at)
            sees = p != 0
            sees |= self.pos <= at
            out[i] = p[sees] @ self.v[sees] if sees.any() else 0.0
            if accumulate:
                self.w += p
        return out

    def evict(self, budget: int, n_first: int, n_recent: int):
        L = len(self.k)
        if L <= budget:
            return
        safe = (self.pos < n_first) | (self.pos >= self.seen - n_recent)
        rank = sorted(range(L), key=lambda t: (not safe[t], np.isnan(self.w[t]),
                                               0.0 if np.isnan(self.w[t]) else -self.w[t], t)
                      if not safe[t] else (False, False, 0.0, t))
        stay = set(rank[:budget])
        movers = iter(sorted(t for t in stay if t >= budget))
        at = [t if t in stay else next(movers) for t in range(budget)]
        self.k, self.v, self.pos, self.w = self.k[at], self.v[at], self.pos[at], self.w[at]
