"""The block-scaled oracle pinned against things other than itself (CPU only)."""

import numpy as np
import pytest
import torch

from oracle import block


def _torch_e4m3(y):
    return torch.as_tensor(y).to(torch.float32).to(torch.float8_e4m3fn).view(torch.uint8).numpy()


def test_e4m3_table_is_the_formats():
    t = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).to(torch.float64).numpy()
    mine = block.e4m3_table()
    assert np.array_equal(np.isnan(t), np.isnan(mine))
    assert np.array_equal(t[~np.isnan(t)], mine[~np.isnan(mine)])
    assert mine[0x7E] == 448 and mine[1] == 2.0 ** -9


def test_e4m3_encode_rounds_to_nearest_even():
    g = np.random.default_rng(0)
    y = np.concatenate([g.standard_normal(20000) * 10.0 ** g.uniform(-4, 2.5, 20000),
                        block._MID, -block._MID, [0.0, -0.0, 448, 463.9]]).astype(np.float32)
    y = np.clip(y, -448, 448)
    assert np.array_equal(block.e4m3_encode(y.astype(np.float64)), _torch_e4m3(y))
    assert block.values(block.e4m3_encode(np.array([1e9, -1e9])), "e4m3").tolist() == [448, -448]


def _pool(kind, gs=16, ps=32, D=8, Hkv=2):
    return block.BlockPool(1, Hkv, D, gs, ps, 4, kind)


@pytest.mark.parametrize("kind,fits", [("int8", 127.5), ("e4m3", 464.0)])
def test_a_scale_doubles_only_when_a_value_does_not_fit(kind, fits):
    s = np.float32(0.037)
    edge = np.float32(fits) * s                      # the largest magnitude that fits
    assert block.grown_scale(s, edge, kind) == (s, 0)
    assert block.grown_scale(s, np.nextafter(edge, np.float32(np.inf)), kind) == (2 * s, 1)
    assert block.grown_scale(s, 8 * edge, kind) == (8 * s, 3)
    assert block.grown_scale(s, np.float32(0), kind) == (s, 0)


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
def test_whole_blocks_are_plain_absmax_quantisation(kind):
    g = np.random.default_rng(1)
    p = _pool(kind)
    x = g.standard_normal((1, 32, 2, 8)).astype(np.float16)
    p.append(0, x, 2 * x, [0], [[2, 1, 0, 3]])
    for h in range(2):
        for b in range(2):
            rows = x[0, 16 * b:16 * b + 16, h].astype(np.float64)
            s = p.k_scales[0, 2, h, b]
            assert abs(s - np.abs(rows).max() / float(block.QMAX[kind])) <= 2.0 ** -24 * s
            back = block.values(p.k_store[0, 2, h, 16 * b:16 * b + 16], kind) * float(s)
            step = 1.0 if kind == "int8" else 32.0
            assert np.abs(back - rows).max() <= (step / 2 + 1e-4) * s
    assert np.array_equal(p.v_scales, 2 * p.k_scales)      # a power of two scales exactly
    assert np.array_equal(p.v_store, p.k_store)


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
def test_growth_keeps_codes_within_one_step(kind):
    """Rows of rising magnitude, one call each: the scale doubles several times, and every
    value stays within a step of the block's last scale (half a step of rounding, and
    half a step for all halvings together)."""
    g = np.random.default_rng(2)
    p = _pool(kind, D=64, Hkv=1)
    x = (g.standard_normal((16, 1, 64)) * 1.3 ** np.arange(16)[:, None, None]).astype(np.float16)
    scales = []
    for i in range(16):
        p.append(0, x[None, i:i + 1], x[None, i:i + 1], [i], [[0]])
        scales.append(float(p.k_scales[0, 0, 0, 0]))
    ratios = np.array(scales[1:]) / np.array(scales[:-1])
    assert set(ratios) <= {1.0, 2.0, 4.0} and (ratios > 1).sum() >= 3
    back = block.values(p.k_store[0, 0, 0, :16], kind) * scales[-1]
    err = np.abs(back - x[:, 0].astype(np.float64))
    if kind == "int8":
        assert err.max() <= 1.0 * scales[-1]
    else:        # relative to the value: 2^-4, plus subnormal halvings of 2^-9 scales
        assert np.all(err <= 2.0 ** -4 * np.abs(x[:, 0]) + 2.0 ** -9 * scales[-1])


def test_halving_rounds_half_to_even():
    p = _pool("int8", D=8, Hkv=1)
    first = np.array([[127, 1, 3, 5, -1, -3, 2, 0]], np.float16)         # scale 1
    p.append(0, first[None, :, None], first[None, :, None], [0], [[0]])
    assert p.k_store[0, 0, 0, 0].tolist() == [127, 1, 3, 5, -1, -3, 2, 0]
    big = np.array([[254, 0, 0, 0, 0, 0, 0, 2]], np.float16)
    p.append(0, big[None, :, None], big[None, :, None], [1], [[0]])
    assert p.k_scales[0, 0, 0, 0] == 2
    assert p.k_store[0, 0, 0, 0].tolist() == [64, 0, 2, 2, 0, -2, 1, 0]
    assert p.k_store[0, 0, 0, 1].tolist() == [127, 0, 0, 0, 0, 0, 0, 1]


def test_zero_blocks_and_bad_places():
    p = _pool("int8")
    z = np.zeros((1, 3, 2, 8), np.float16)
    p.append(0, z, z, [0], [[1]])
    assert not p.k_scales.any() and not p.k_store.any()
    one = np.ones((1, 1, 2, 8), np.float16)
    p.append(0, one, one, [3], [[1]])                   # a zero scale is set afresh
    assert np.all(p.k_scales[0, 1, :, 0] == np.float32(1) / np.float32(127))
    assert np.all(p.k_store[0, 1, :, 3] == 127) and not p.k_store[0, 1, :, :3].any()
    before = p.k_store.copy()
    p.append(0, one, one, [40], [[1]])                  # beyond the row
    p.append(0, one, one, [-1], [[1]])                  # a negative position
    p.append(0, one, one, [4], [[7]])                   # no such page
    assert np.array_equal(before, p.k_store)
