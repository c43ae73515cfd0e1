"""Oracle: attention with shaped scores, in fp64 (test infrastructure only).

Query i of Q sits at P = length - Q + i; its score with position p, s = scale (q . k), becomes
cap tanh(s / cap) (cap 0: s), then s + slope_h (p - P).  It attends p < length with p < prefix, or
p <= P and (window > 0) p > P - window.  A query at a negative position yields 0.
"""

import math

import numpy as np


def seen(length, Q, window=0, prefix=0):
    """bool [Q][length]: which positions each query attends."""
    p = np.arange(length)[None, :]
    P = length - Q + np.arange(Q)[:, None]
    near = (p <= P) & ((p > P - window) if window > 0 else True)
    return (near | (p < prefix)) & (P >= 0)


def attention(q16, khat, vhat, length, window=0, cap=0.0, slopes=None, prefix=0, scale=None):
    """q16: fp16 [Q][H][D]; khat, vhat: fp64 [>= length][Hkv][D] -> fp64 [Q][H][D]."""
    q = np.asarray(q16, np.float16).astype(np.float64)
    Q, H, D = q.shape
    G = H // khat.shape[1]
    sc = 1.0 / math.sqrt(D) if scale is None else float(scale)
    look = seen(length, Q, window, prefix)
    away = np.arange(length)[None, :] - (length - Q + np.arange(Q))[:, None]
    out = np.zeros((Q, H, D))
    for h in range(H):
        s = sc * (q[:, h] @ khat[:length, h // G].T)
        if cap:
            s = cap * np.tanh(s / cap)
        if slopes is not None:
            s = s + float(slopes[h]) * away
        s = np.where(look, s, -np.inf)
        for i in range(Q):
            if look[i].any():
                w = np.exp(s[i] - s[i].max())
                out[i, h] = (w / w.sum()) @ np.where(look[i][:, None], vhat[:length, h // G], 0.0)
    return out
