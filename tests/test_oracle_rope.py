"""The oracles of rotated appends and draft verification against plain statements of the same."""

from fractions import Fraction

import numpy as np
import pytest

from oracle import block, pool, rope, verify


@pytest.mark.parametrize("style", ["halves", "pairs"])
@pytest.mark.parametrize("R", [16, 48, 64])
def test_turns_are_complex_products(style, R):
    """fp32: two products and a sum, each off by half a step of a value of at most
    |a| + |b|: 3 * 2^-24 (|a| + |b|)."""
    g = np.random.default_rng(R)
    x = g.standard_normal((5, 3, 64)).astype(np.float16)
    at = g.integers(0, 1000, (5, R // 2))
    tab = rope.table(1000, R)
    got, want = rope.turn(x, tab, at, style), rope.turn64(x, tab, at, style)
    assert np.abs(got - want).max() <= 3 * 2.0 ** -24 * 2 * np.abs(x.astype(np.float64)).max()
    assert np.array_equal(got[..., R:], x[..., R:])
    norm = np.linalg.norm(want, axis=-1)
    assert np.allclose(norm, np.linalg.norm(x.astype(np.float64), axis=-1), rtol=1e-6)


def test_scores_depend_on_the_distance_alone():
    g = np.random.default_rng(0)
    q, k = g.standard_normal((2, 1, 1, 64)).astype(np.float16)
    tab = rope.table(2000, 64)
    dot = [float((rope.turn64(q, tab, np.full((1, 32), p), "halves")
                  * rope.turn64(k, tab, np.full((1, 32), p - 100), "halves")).sum())
           for p in (100, 700, 1999)]
    # the table's fp32 values are off by 2^-25 each, 64 products of about 1
    assert np.ptp(dot) <= 4 * 64 * 2.0 ** -25 * 8


def test_positions_by_axis_and_outside_the_table():
    at = rope.rows_of(7, 2, [[1, 2], [30, 31], [500, 501]], [0, 0, 1, 1, 2, 2, 0, 1], R=16)
    assert at.tolist() == [[1, 1, 30, 30, 500, 500, 1, 30], [2, 2, 31, 31, 501, 501, 2, 31]]
    assert rope.rows_of(7, 2, R=16).tolist() == [[7] * 8, [8] * 8]
    x = np.ones((1, 1, 16), np.float16)
    tab = rope.table(10, 16)
    out = rope.turn(x, tab, np.array([[3, 3, 3, 3, 10, -1, 3, 3]]), "pairs")
    assert np.array_equal(out[0, 0, 8:12], [1, 1, 1, 1]) and not np.array_equal(out[0, 0, :2], [1, 1])


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
def test_unturned_appends_are_the_pools_own(kind):
    g = np.random.default_rng(1)
    k, v = g.standard_normal((2, 1, 40, 2, 64)).astype(np.float16)
    a, b = (block.BlockPool(1, 2, 64, 16, 16, 4, kind) for _ in range(2))
    row = np.array([2, 0, 3])
    a.append(0, k, v, [3], row[None])
    rope.append(b, 0, k[0].astype(np.float32), v[0], 3, row)
    for name in ("k_store", "v_store", "k_scales", "v_scales"):
        assert np.array_equal(getattr(a, name), getattr(b, name))


@pytest.mark.parametrize("variant", [pool.K8V8, pool.K8V16, pool.K16V8, pool.K8V4, pool.Q4_0])
def test_unturned_appends_are_the_row_pools_own(variant):
    g = np.random.default_rng(2)
    k, v = g.standard_normal((2, 20, 2, 64)).astype(np.float16)
    a, b = (pool.Pool(1, 2, 64, 32, 16, 4, variant) for _ in range(2))
    row = np.array([2, 0, 3])
    a.append_contiguous(0, k, v, 3, row)
    rope.append(b, 0, k.astype(np.float32), v, 3, row)
    for name in ("k_store", "v_store", "k_scales", "v_scales"):
        x, y = getattr(a, name), getattr(b, name)
        assert x is None and y is None or np.array_equal(x, y)


def test_verification_draws_the_targets_tokens():
    """Summed over all drafts and numbers, a token comes out as often as the target has it: drafts
    of probability q(x), taken with min(1, p / q), and what is left drawn by p - q."""
    p, q = np.array([0.5, 0.25, 0.125, 0.125], np.float32), np.array([0.125, 0.25, 0.5, 0.125],
                                                                    np.float32)
    n, grid = 64, (np.arange(64) + 0.5).astype(np.float32) / 64
    share = [Fraction(0)] * 4
    for x in range(4):
        for u in grid:
            for s in grid:
                t, v = verify.one(np.stack([p, p]), q[None], [x], [u], s)
                share[x if t else v] += Fraction(float(q[x])) / (n * n)
    assert [float(f) for f in share] == pytest.approx(p.tolist(), abs=1 / 64)


def test_verification_by_hand():
    p = np.array([[0.5, 0.5, 0, 0], [0.25, 0.25, 0.25, 0.25], [0, 0, 0, 1]], np.float32)
    q = np.array([[0.5, 0.25, 0.25, 0], [1, 0, 0, 0]], np.float32)
    assert verify.one(p, q, [0, 0], [0.9, 0.2], 0.5) == (2, 3)
    assert verify.one(p, q, [0, 0], [0.9, 0.25], 0.0) == (1, 1)       # 0.25 * 1 < 0.25 is not so
    assert verify.one(p, q, [0, 0], [0.9, 0.25], 0.999) == (1, 3)
    assert verify.one(p, q, [2, 0], [0.0, 0.0], 0.5) == (0, 1)        # nothing but token 1 is left
    assert verify.one(p, None, [0, 3], [0.4, 0.3], 0.4) == (1, 1)     # token 3 refused and left out
    assert verify.one(p[:1], None, [], [], 0.5) == (0, 1)
    assert verify.one(p[:2], p[:1], [2], [0.5], 0.1) == (0, 0)        # p = q: by p itself
    assert verify.one(0 * p[:1], None, [], [], 0.5) == (0, -1)
