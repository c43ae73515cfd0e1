"""The oracle of shaped scores against the plain one and against its statement, one pair at a time."""

import math

import numpy as np
import pytest

from oracle import attention as oatt
from oracle import scored


def _rows(n, H, Hkv, D, Q, seed=0):
    g = np.random.default_rng(seed)
    return (g.standard_normal((Q, H, D)).astype(np.float16), g.standard_normal((n, Hkv, D)),
            g.standard_normal((n, Hkv, D)))


def test_unshaped_scores_are_plain_attention():
    q, k, v = _rows(40, 4, 2, 64, 5)
    got = scored.attention(q, k, v, 40)
    assert np.allclose(got, oatt.prefill_chunk(q, k, v, 35), rtol=1e-12, atol=1e-14)
    got = scored.attention(q[:1], k, v, 40, window=7)
    assert np.allclose(got[0], oatt.decode(q[0], k, v, 40, 7), rtol=1e-12, atol=1e-14)


@pytest.mark.parametrize("window,prefix", [(0, 0), (0, 38), (6, 0), (6, 3), (6, 39), (1, 100)])
def test_by_hand(window, prefix):
    n, Q, H, D, cap = 40, 3, 2, 64, 2.0
    q, k, v = _rows(n, H, 1, D, Q, 1)
    slopes = [0.25, 0.5]
    got = scored.attention(q, k, v, n, window, cap, slopes, prefix)
    for i in range(Q):
        P = n - Q + i
        at = [p for p in range(n) if p < prefix or (p <= P and (not window or P - p < window))]
        for h in range(H):
            w = [math.exp(cap * math.tanh(float(q[i, h].astype(float) @ k[p, 0]) / 8 / cap)
                          + slopes[h] * (p - P)) for p in at]
            want = sum(a * v[p, 0] for a, p in zip(w, at)) / sum(w)
            assert np.allclose(got[i, h], want, rtol=1e-12, atol=1e-14)


def test_queries_before_the_start():
    q, k, v = _rows(2, 1, 1, 64, 4)
    got = scored.attention(q, k, v, 2, prefix=5)
    assert not got[:2].any() and got[2:].all()
    assert np.allclose(got[2], got[2])
