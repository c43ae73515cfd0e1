"""Oracle: verification of drafted tokens (test infrastructure only), in whole numbers.

Probabilities are taken into [0, 1] (NaN: 0); a draft is taken while u q(x) < p(x) as fractions; in the
weights a probability is p * 2^60 rounded to a whole number; the token behind the drafts taken is the lowest v whose weights
0 .. v sum to more than u times all weights.
"""

from fractions import Fraction

import numpy as np

ONE = 1 << 60


def fixed(p):
    """fp32 array -> whole multiples of 2^-60 (exact in fp64: 24 bits and a power of two)."""
    p = np.nan_to_num(np.asarray(p, np.float32).astype(np.float64), nan=0.0)
    return np.rint(np.clip(p, 0.0, 1.0) * 2.0 ** 60).astype(np.uint64)


def nearest(p):
    """An fp32 number as the nearest of [0, 1] (NaN: 0)."""
    return Fraction(0) if np.isnan(p) else Fraction(min(max(float(p), 0.0), 1.0))


def one(target, draft, x, u, sample_u):
    """One sequence: target [n + 1][V], draft [n][V] or None, x [n], u [n] -> (taken, token)."""
    V, n = target.shape[1], len(x)
    taken = 0
    while taken < n:
        v = int(x[taken])
        if not 0 <= v < V:
            break
        q = Fraction(1) if draft is None else nearest(draft[taken, v])
        p = nearest(target[taken, v])
        if np.isnan(u[taken]) or not Fraction(float(u[taken])) * q < p:
            break
        taken += 1
    p = fixed(target[taken])
    w = p.copy()
    if taken < n:
        if draft is not None:
            q = fixed(draft[taken])
            w = np.where(p > q, p - q, np.uint64(0))
        elif 0 <= x[taken] < V:
            w[int(x[taken])] = 0
    if not w.any():
        w = p
    if not w.any():
        return taken, -1
    c = np.cumsum(w, dtype=np.uint64)
    su = 0.0 if np.isnan(sample_u) else min(max(float(sample_u), 0.0), 1.0 - 2.0 ** -24)
    place = (int(fixed(su)) << 4) * int(c[-1]) >> 64
    return taken, int(np.searchsorted(c, np.uint64(place), side="right"))


def batch(target, draft, x, u, sample_u, n_drafts=None, seq_lens=None):
    """(tokens [B][n + 1], n_accepted [B], seq_lens [B] or None) of a call."""
    B, n = x.shape
    tokens = np.full((B, n + 1), -1, np.int32)
    acc = np.zeros(B, np.int32)
    lens = None if seq_lens is None else np.array(seq_lens, np.int32)
    for b in range(B):
        k = n if n_drafts is None else min(int(n_drafts[b]), n)
        if k < 0:
            continue
        t, v = one(target[b, :k + 1], None if draft is None else draft[b, :k], x[b, :k], u[b, :k],
                   sample_u[b])
        tokens[b, :t], tokens[b, t], acc[b] = x[b, :t], v, t
        if lens is not None:
            lens[b] -= k - t
    return tokens, acc, lens
