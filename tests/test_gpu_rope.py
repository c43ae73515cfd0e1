"""Rotated appends on the GPU, bit for bit: every operation is rounded by itself, so that queries,
codes and scales are the oracle's."""

import numpy as np
import pytest
import torch

from int8_kv_cache_02_gb300 import inputs
from oracle import pool as opool
from oracle import rope
from tests import block_util as bu
from tests import gpu_util as gu

pytestmark = pytest.mark.gpu

KINDS = ["int8", "e4m3"]


def _dev(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _rows(g, S, n, H, Hkv, D):
    k = torch.randn((S, n, Hkv, D), generator=g)
    k[..., :4] *= 20
    q, v = (torch.randn((S, n, h, D), generator=g).half() for h in (H, Hkv))
    return q, k.half(), v


def _oracle(orc, q, k, v, pos, pt, tab, style, lens=None, positions=None, pair_axis=None):
    """The oracle's pool after the call -> the queries it gives, zeros behind lens."""
    S, n = k.shape[:2]
    out = np.zeros(q.shape, np.float16)
    for b in range(S):
        m = n if lens is None else min(max(lens[b], 0), n)
        at = rope.rows_of(pos[b], n, None if positions is None else positions[:, b].numpy(),
                          None if pair_axis is None else pair_axis.numpy(), tab.shape[1])[:m]
        out[b, :m] = rope.turn(q[b, :m].numpy(), tab, at, style).astype(np.float16)
        rope.append(orc, 0, rope.turn(k[b, :m].numpy(), tab, at, style), v[b, :m].numpy(), pos[b],
                    pt[b].numpy())
    return out


def _call(dev, q, k, v, pos, pt, tab, style="halves", lens=None, positions=None, pair_axis=None,
          q_out=None):
    from int8_kv_cache_02_gb300 import binding
    q_out = torch.zeros(q.shape, dtype=torch.float16, device="cuda") if q_out is None else q_out
    binding.kv_rope_append(dev, 0, k.cuda(), v.cuda(), _dev(pos), pt.cuda(),
                           torch.from_numpy(tab).cuda(), q=q.cuda(), q_out=q_out, style=style,
                           positions=None if positions is None else positions.cuda(),
                           pair_axis=pair_axis, new_lens=None if lens is None else _dev(lens))
    torch.cuda.synchronize()
    return q_out.cpu().numpy()


def _same(a, b):
    assert np.array_equal(a.view(np.uint16), b.view(np.uint16))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("style", ["halves", "pairs"])
@pytest.mark.parametrize("D,R,gs,ps,n", [(64, 64, 16, 16, 1), (64, 16, 16, 32, 9), (64, 48, 64, 64, 70),
                                         (128, 128, 64, 64, 1), (128, 80, 32, 64, 40),
                                         (128, 128, 128, 128, 131), (256, 256, 64, 64, 3),
                                         (256, 64, 128, 128, 140), (256, 256, 16, 16, 33)])
def test_block_pools(kind, style, D, R, gs, ps, n):
    """A prompt behind an odd place, then the same positions' successors: blocks that hold rows."""
    g = torch.Generator().manual_seed(D + R + n)
    pos = [0, 5, gs, 2 * gs - 1]
    pt, n_pages = inputs.page_table([p + 2 * n for p in pos], ps, seed=1)
    dev, orc = bu.make_pools(kind, 3, D, gs, ps, n_pages)
    tab = rope.table(pos[-1] + 2 * n, R)
    for step in range(2):
        q, k, v = _rows(g, 4, n, 6, 3, D)
        k = k * 3.0 ** step
        want = _oracle(orc, q, k, v, pos, pt, tab, style)
        _same(_call(dev, q, k, v, pos, pt, tab, style), want)
        bu.assert_same(dev, orc, f"step {step}")
        pos = [p + n for p in pos]
    from int8_kv_cache_02_gb300 import binding
    assert binding.kv_pool_read_device_error(dev) == 0


@pytest.mark.parametrize("variant", [opool.K8V8, opool.K8V16, opool.K16V8, opool.K8V4, opool.Q4_0])
@pytest.mark.parametrize("style", ["halves", "pairs"])
@pytest.mark.parametrize("D,R,gs,n", [(64, 64, 64, 3), (64, 32, 16, 17), (128, 112, 32, 5),
                                      (128, 128, 128, 1), (256, 64, 64, 7), (256, 256, 256, 2)])
def test_row_pools(variant, style, D, R, gs, n):
    gu.lib_ready()
    g = torch.Generator().manual_seed(D + R + n)
    pos = [0, 31, 62]
    pt, n_pages = inputs.page_table([p + n for p in pos], 32, seed=1)
    dev, orc = gu.make_pools(1, 2, D, gs, 32, n_pages, variant)
    tab = rope.table(pos[-1] + n, R)
    q, k, v = _rows(g, 3, n, 10, 2, D)
    want = _oracle(orc, q, k, v, pos, pt, tab, style)
    _same(_call(dev, q, k, v, pos, pt, tab, style), want)
    gu.regions_equal(dev, orc)


@pytest.mark.parametrize("kind", KINDS + ["rows"])
@pytest.mark.parametrize("style", ["halves", "pairs"])
@pytest.mark.parametrize("blend", [False, True])
def test_axes_and_ragged_sequences(kind, style, blend):
    """Three axes in runs of pairs, and in turn (`blend`); sequences of none, some and all tokens, and
    of more than there are; rows of q_out behind them stay as they were."""
    from int8_kv_cache_02_gb300 import binding
    g = torch.Generator().manual_seed(5)
    S, n, D, R = 5, 21, 128, 96
    pos, lens = [3, 0, 40, 7, 64], [21, 0, 8, -2, 25]
    pt, n_pages = inputs.page_table([p + n for p in pos], 64, seed=3)
    if kind == "rows":
        gu.lib_ready()
        dev, orc = gu.make_pools(1, 2, D, 64, 64, n_pages, opool.K8V8)
    else:
        dev, orc = bu.make_pools(kind, 2, D, 32, 64, n_pages)
    tab = rope.table(300, R)
    axis = torch.arange(R // 2)
    axis = (axis % 3 if blend else 3 * axis // (R // 2)).to(torch.uint8)
    positions = torch.randint(0, 300, (3, S, n), generator=g, dtype=torch.int32)
    q, k, v = _rows(g, S, n, 4, 2, D)
    want = _oracle(orc, q, k, v, pos, pt, tab, style, lens, positions, axis)
    before = torch.full(q.shape, 7.0, dtype=torch.float16, device="cuda")
    got = _call(dev, q, k, v, pos, pt, tab, style, lens, positions, axis, q_out=before)
    for b in range(S):
        m = min(max(lens[b], 0), n)
        _same(got[b, :m], want[b, :m])
        assert (got[b, m:] == 7.0).all()
    (gu.regions_equal if kind == "rows" else bu.assert_same)(dev, orc)
    assert binding.kv_pool_read_device_error(dev) == binding.DEVERR_LENGTH      # 25 of 21 tokens


@pytest.mark.parametrize("kind", KINDS + ["rows"])
def test_parts_of_a_projection_and_in_place(kind):
    """q, k and v inside one projection's rows; then q_out is q; and no queries at all."""
    from int8_kv_cache_02_gb300 import binding
    g = torch.Generator().manual_seed(6)
    S, n, H, Hkv, D = 3, 19, 8, 2, 64
    pos = [0, 9, 30]
    pt, n_pages = inputs.page_table([p + n for p in pos], 32, seed=3)
    tab = rope.table(64, D)
    both = []
    for _ in range(3):
        if kind == "rows":
            gu.lib_ready()
            both.append(gu.make_pools(1, Hkv, D, D, 32, n_pages, opool.K8V8))
        else:
            both.append(bu.make_pools(kind, Hkv, D, 16, 32, n_pages))
    q, k, v = _rows(g, S, n, H, Hkv, D)
    wide = torch.cat([q, k, v], dim=2).cuda()
    same = gu.regions_equal if kind == "rows" else bu.assert_same
    dt = torch.from_numpy(tab).cuda()
    dev, orc = both[0]
    want = _oracle(orc, q, k, v, pos, pt, tab, "halves")
    out = torch.empty(q.shape, dtype=torch.float16, device="cuda")
    binding.kv_rope_append(dev, 0, wide[:, :, H:H + Hkv], wide[:, :, H + Hkv:], _dev(pos), pt.cuda(),
                           dt, q=wide[:, :, :H], q_out=out)
    _same(out.cpu().numpy(), want)
    same(dev, orc)
    dev = both[1][0]
    mine = q.cuda()
    binding.kv_rope_append(dev, 0, k.cuda(), v.cuda(), _dev(pos), pt.cuda(), dt, q=mine, q_out=mine)
    _same(mine.cpu().numpy(), want)
    same(dev, orc)
    dev = both[2][0]
    binding.kv_rope_append(dev, 0, k.cuda(), v.cuda(), _dev(pos), pt.cuda(), dt)
    same(dev, orc)


@pytest.mark.parametrize("kind", KINDS + ["rows"])
def test_tokens_without_a_place(kind):
    """Negative positions, rows that are too short, pages that are none, positions outside the table:
    flagged and left out (keys) or not turned (queries)."""
    from int8_kv_cache_02_gb300 import binding
    g = torch.Generator().manual_seed(7)
    n, D = 12, 64
    pos = [-5, 58, 16, 0]
    pt = torch.tensor([[0, 1, 2, 3], [4, 5, 6, 7], [8, -1, 99, 9], [10, 11, 12, 13]],
                      dtype=torch.int32)
    if kind == "rows":
        gu.lib_ready()
        dev, orc = gu.make_pools(1, 2, D, D, 16, 14, opool.K8V8)
    else:
        dev, orc = bu.make_pools(kind, 2, D, 16, 16, 14)
    tab = rope.table(66, D)
    q, k, v = _rows(g, 4, n, 2, 2, D)
    want = _oracle(orc, q, k, v, pos, pt, tab, "halves")
    _same(_call(dev, q, k, v, pos, pt, tab), want)
    (gu.regions_equal if kind == "rows" else bu.assert_same)(dev, orc)
    assert binding.kv_pool_read_device_error(dev) == binding.DEVERR_LENGTH | binding.DEVERR_PAGE_ID


@pytest.mark.parametrize("kind", KINDS + ["rows"])
@pytest.mark.parametrize("n", [2, 5, 17, 40])
def test_positions_at_the_ends_of_int32(kind, n):
    """INT32_MIN and its successors, whose distance to a block's first token is beyond 32 bits; INT32_MAX;
    one sequence among them that has a place."""
    from int8_kv_cache_02_gb300 import binding
    g = torch.Generator().manual_seed(n)
    D, pos = 64, [-2 ** 31, 3, 2 ** 31 - 1, -2 ** 31 + 1, -2 ** 31 + n, 2 ** 31 - n]
    pt = torch.arange(24, dtype=torch.int32).view(6, 4)
    if kind == "rows":
        gu.lib_ready()
        dev, orc = gu.make_pools(1, 2, D, D, 16, 24, opool.K8V8)
    else:
        dev, orc = bu.make_pools(kind, 2, D, 16, 16, 24)
    tab = rope.table(60, D)
    q, k, v = _rows(g, 6, n, 2, 2, D)
    want = _oracle(orc, q, k, v, pos, pt, tab, "halves")
    _same(_call(dev, q, k, v, pos, pt, tab), want)
    (gu.regions_equal if kind == "rows" else bu.assert_same)(dev, orc)
    assert binding.kv_pool_read_device_error(dev) == binding.DEVERR_LENGTH


@pytest.mark.parametrize("kind", KINDS + ["rows", "q4_0"])
def test_sequences_without_tokens_are_no_error(kind):
    """Entries that pad a batch: any position and page table row, no tokens.  Nothing is flagged, and the
    others' rows are there."""
    from int8_kv_cache_02_gb300 import binding
    g = torch.Generator().manual_seed(16)
    n, D = 5, 64
    pos, lens = [-1, 3, -2 ** 31, 2 ** 31 - 1, 10 ** 6, 0], [0, 5, 0, 0, -3, 2]
    pt = torch.tensor([[-1, -1], [0, 1], [99, 99], [-1, -1], [-7, -1], [2, 3]], dtype=torch.int32)
    if kind in KINDS:
        dev, orc = bu.make_pools(kind, 2, D, 16, 16, 4)
    else:
        gu.lib_ready()
        dev, orc = gu.make_pools(1, 2, D, D, 16, 4, opool.K8V8 if kind == "rows" else opool.Q4_0)
    tab = rope.table(40, D)
    q, k, v = _rows(g, 6, n, 2, 2, D)
    want = _oracle(orc, q, k, v, pos, pt, tab, "halves", lens)
    got = _call(dev, q, k, v, pos, pt, tab, lens=lens)
    for b in (1, 5):
        _same(got[b, :lens[b]], want[b, :lens[b]])
    (bu.assert_same if kind in KINDS else gu.regions_equal)(dev, orc)
    assert binding.kv_pool_read_device_error(dev) == 0


@pytest.mark.parametrize("kind", KINDS)
def test_scales_from_tiny_products(kind):
    """A sine of 2^-110 leaves keys whose scale has no reciprocal in fp32; zeros leave scale 0."""
    k = torch.zeros((1, 3, 1, 64), dtype=torch.float16)
    k[0, 0, 0, 32:40] = torch.tensor([1, 2, 3, 4, 5, 6, 7, 127.0]).half()
    tab = np.zeros((3, 64), np.float32)
    tab[:, 32:] = 2.0 ** -110
    tab[1:, 32:] = 2.0 ** -104      # (a block that grows)
    pt = torch.zeros((1, 1), dtype=torch.int32)
    dev, orc = bu.make_pools(kind, 1, 64, 16, 16, 1)
    k[0, 2] = k[0, 0]
    for i in range(3):
        one = k[:, i:i + 1]
        want = _oracle(orc, one, one, one, [i], pt, tab, "halves")
        _same(_call(dev, one, one, one, [i], pt, tab), want)
        bu.assert_same(dev, orc, f"token {i}")


@pytest.mark.parametrize("n", [1, 300])
def test_many_query_heads_and_tokens(n):
    """Threads that take several heads, an uneven number of them."""
    g = torch.Generator().manual_seed(n)
    S, H, D = (200, 21, 128) if n == 1 else (9, 13, 128)
    pos = list(range(S))
    pt, n_pages = inputs.page_table([p + n for p in pos], 64, seed=3)
    dev, orc = bu.make_pools("int8", 1, D, 64, 64, n_pages)
    tab = rope.table(S + n, D)
    q, k, v = _rows(g, S, n, H, 1, D)
    want = _oracle(orc, q, k, v, pos, pt, tab, "halves")
    _same(_call(dev, q, k, v, pos, pt, tab), want)
    bu.assert_same(dev, orc)


@pytest.mark.parametrize("kind", KINDS + ["rows"])
def test_layers_and_pages_past_4_gb(kind):
    """The second layer's last pages, more than 2^32 bytes into either store; what comes to lie there is
    what a small pool gets, the first layer stays as it was, and shaped scores read it back."""
    from int8_kv_cache_02_gb300 import binding as b
    g = torch.Generator().manual_seed(9)
    D, ps, n_pages, n = 256, 128, 72000, 150
    variant = {"int8": "k8v8_block", "e4m3": "f8_block", "rows": "k8v8"}[kind]
    gs = 256 if kind == "rows" else 32
    far = b.KVPool(2, 1, D, gs, ps, n_pages, variant)
    near = b.KVPool(1, 1, D, gs, ps, 2, variant)
    assert far.k_store[1].numel() * 2 > 1 << 32
    q, k, v = (t.cuda() for t in _rows(g, 1, n, 8, 1, D))
    tab = torch.from_numpy(rope.table(n, D)).cuda()
    out = [torch.empty_like(q) for _ in range(2)]
    ft, nt = _dev([[n_pages - 1, n_pages - 2]]), _dev([[0, 1]])
    for pool, layer, table, o in ((far, 1, ft, out[0]), (near, 0, nt, out[1])):
        b.kv_rope_append(pool, layer, k, v, _dev([0]), table, tab, q=q, q_out=o)
    assert torch.equal(out[0], out[1])
    for name in ("k_store", "v_store", "k_scales", "v_scales"):
        x, y = (getattr(p, name).view(torch.uint8) for p in (far, near))
        assert torch.equal(x[1, [n_pages - 1, n_pages - 2]], y[0])
        assert not x[0, -4:].any() and not x[1, -6:-2].any()
    if kind == "rows":
        return
    lens = _dev([n])
    got = [torch.empty((1, 4, 8, D), device="cuda") for _ in range(2)]
    chunk = [torch.empty((n, 8, D), device="cuda") for _ in range(2)]
    for pool, layer, table, o, c in ((far, 1, ft, got[0], chunk[0]), (near, 0, nt, got[1], chunk[1])):
        b.attn_decode_scored_int8(pool, layer, q[:, -4:].contiguous(), lens, table, o, None,
                                  softcap=20.0, n_splits=1)
        b.attn_prefill_chunk_scored_int8(pool, layer, q[0], 0, table[0], c, None, softcap=20.0,
                                         n_splits=1)
    assert got[0].any() and torch.equal(got[0], got[1]) and torch.equal(chunk[0], chunk[1])
    assert b.kv_pool_read_device_error(far) == 0


def test_replayed_on_another_stream():
    """Captured once, replayed as positions and lengths move on, on a stream of its own."""
    from int8_kv_cache_02_gb300 import binding
    g = torch.Generator().manual_seed(8)
    S, n, D = 2, 3, 128
    pt, n_pages = inputs.page_table([64, 64], 32, seed=3)
    dev, orc = bu.make_pools("e4m3", 2, D, 32, 32, n_pages)
    tab = rope.table(64, D)
    q, k, v = (torch.zeros((S, n, h, D), dtype=torch.float16, device="cuda") for h in (4, 2, 2))
    pos, lens, out = _dev([0, 0]), _dev([n, n]), torch.zeros_like(q)
    args = (pt.cuda(), torch.from_numpy(tab).cuda())
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(stream):
        binding.kv_rope_append(dev, 0, k, v, pos, *args, q=q, q_out=out, new_lens=_dev([0, 0]))
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=stream):
            binding.kv_rope_append(dev, 0, k, v, pos, *args, q=q, q_out=out, new_lens=lens)
        at = [0, 5]
        for step in range(4):
            m = [3, step]
            hq, hk, hv = _rows(g, S, n, 4, 2, D)
            want = _oracle(orc, hq, hk, hv, at, pt, tab, "halves", m)
            for t, h in ((q, hq), (k, hk), (v, hv), (pos, torch.tensor(at)),
                         (lens, torch.tensor(m))):
                t.copy_(h)
            graph.replay()
            stream.synchronize()
            for b in range(S):
                _same(out[b, :m[b]].cpu().numpy(), want[b, :m[b]])
            bu.assert_same(dev, orc, f"step {step}")
            at = [a + x for a, x in zip(at, m)]
