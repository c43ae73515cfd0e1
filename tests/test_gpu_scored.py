"""Attention with shaped scores on the GPU, against fp64."""

import math

import numpy as np
import pytest
import torch

from int8_kv_cache_02_gb300 import inputs
from oracle import rope, scored, verify
from tests import block_util as bu

pytestmark = pytest.mark.gpu

KINDS = ["int8", "e4m3"]


def _dev(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _filled(kind, seed, lens, Hkv, D, gs, ps, size=1.0):
    g = torch.Generator().manual_seed(seed)
    pt, n_pages = inputs.page_table([max(n, 1) for n in lens], ps, seed=seed)
    dev, orc = bu.make_pools(kind, Hkv, D, gs, ps, n_pages)
    for b, n in enumerate(lens):
        if n > 0:
            k, v = (torch.randn((1, n, Hkv, D), generator=g) for _ in range(2))
            bu.append(dev, orc, 0, (size * k).half(), v.half(), [0], pt[b:b + 1])
    return g, pt, dev, orc


def _slopes(H):
    return (2.0 ** (-8.0 * torch.arange(1, H + 1) / H)).float()


def _reference(orc, q, lens, pt, windows=0, cap=0.0, slopes=None, prefixes=None, scale=None):
    out = np.zeros(q.shape)
    for b, n in enumerate(lens):
        if n > 0:
            kh, vh = orc.gather(0, pt[b].numpy(), n)
            out[b] = scored.attention(q[b].numpy(), kh, vh, n, windows, cap,
                                      None if slopes is None else slopes.numpy(),
                                      0 if prefixes is None else prefixes[b], scale)
    return out


def _decode(dev, q, lens, pt, window=0, cap=0.0, slopes=None, prefixes=None, n_splits=0, scale=0.0):
    from int8_kv_cache_02_gb300 import binding
    B, Q, H, D = q.shape
    ws = dev.decode_workspace(B * Q, H, n_splits or 256)
    ws.fill_(0xFF)
    out = torch.full(q.shape, float("nan"), dtype=torch.float32, device="cuda")
    args = (q.cuda(), _dev(lens), pt.cuda(), out) if Q > 1 else \
        (q[:, 0].contiguous().cuda(), _dev(lens), pt.cuda(), out[:, 0].view(B, H, D))
    binding.attn_decode_scored_int8(dev, 0, *args, ws, window=window, softcap=cap,
                                    slopes=None if slopes is None else slopes.cuda(),
                                    prefix_lens=None if prefixes is None else _dev(prefixes),
                                    softmax_scale=scale, n_splits=n_splits)
    torch.cuda.synchronize()
    return out.cpu().numpy()


def _chunk(dev, q, start, row, window=0, cap=0.0, slopes=None, prefix=0, n_splits=0, scale=0.0):
    from int8_kv_cache_02_gb300 import binding
    n_new, H, D = q.shape
    near = min(start, window + prefix) if window else start
    ns = n_splits or binding.attn_prefill_n_splits(dev, n_new, H, near)
    n = binding.attn_prefill_workspace_bytes(n_new, H, dev.n_kv_heads, D, ns)
    ws = torch.full((max(n, 16),), 255, dtype=torch.uint8, device="cuda")
    out = torch.full(q.shape, float("nan"), device="cuda")
    binding.attn_prefill_chunk_scored_int8(dev, 0, q.cuda(), start, row.cuda(), out, ws,
                                           window=window, softcap=cap,
                                           slopes=None if slopes is None else slopes.cuda(),
                                           prefix_len=prefix, softmax_scale=scale, n_splits=n_splits)
    torch.cuda.synchronize()
    return out.cpu().numpy()


# Scores here stay within 8 in base 2 (a cap only lowers them).  The cap's arithmetic is off by
# 1.3 * 2^-24 of a score and the bias adds two roundings of values that stay below 40 where a weight
# is above 2^-40: as much again as assert_close grants a plain score of 8, so z_max is 16.
Z = 16.0

SHAPES = [dict(cap=30.0), dict(cap=2.0, slopes=True), dict(slopes=True), dict(window=37),
          dict(window=100, prefixes=True, cap=4.0), dict(prefixes=True, slopes=True),
          dict(window=1, prefixes=True), dict(window=300, prefixes=True, slopes=True, cap=50.0)]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("shape", range(len(SHAPES)))
@pytest.mark.parametrize("D,Hkv,G,ps,gs,Q", [(64, 1, 8, 16, 16, 1), (64, 2, 3, 64, 32, 5),
                                             (128, 2, 4, 64, 64, 1), (128, 1, 4, 32, 16, 4),
                                             (128, 3, 1, 128, 128, 2), (256, 2, 8, 64, 64, 1),
                                             (256, 1, 2, 64, 32, 9)])
def test_decode(kind, shape, D, Hkv, G, ps, gs, Q):
    """Ragged lengths (none, one, a tile's ends, long), prefixes of none, some and all positions, every
    schedule."""
    from int8_kv_cache_02_gb300 import binding
    lens = [0, 1, 16, 17, 333, 64, 900, 5]
    g, pt, dev, orc = _filled(kind, D + Q, lens, Hkv, D, gs, ps)
    s = dict(SHAPES[shape])
    slopes = _slopes(Hkv * G) if s.pop("slopes", False) else None
    prefixes = [3, 1, 16, 4, 50, -7, 33, 1000] if s.pop("prefixes", False) else None
    q = torch.randn((8, Q, Hkv * G, D), generator=g).half()
    ref = _reference(orc, q, lens, pt, s.get("window", 0), s.get("cap", 0.0), slopes, prefixes)
    for n_splits in (0, 1, 2, 3, 8, 40):
        got = _decode(dev, q, lens, pt, slopes=slopes, prefixes=prefixes, n_splits=n_splits, **s)
        bu.assert_close(got, ref, z_max=Z, what=f"{n_splits} splits")
    assert binding.kv_pool_read_device_error(dev) == 0


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("Q,G", [(16, 4), (64, 1), (64, 8), (3, 8)])
def test_long_windows_of_queries(kind, Q, G):
    lens = [Q, Q - 1, 200, 0, 2]
    g, pt, dev, orc = _filled(kind, Q + G, lens, 2, 128, 16, 16)
    q = torch.randn((5, Q, 2 * G, 128), generator=g).half()
    slopes, prefixes = _slopes(2 * G), [5, 200, 20, 3, 2]
    ref = _reference(orc, q, lens, pt, 30, 10.0, slopes, prefixes)
    for n_splits in (0, 1, 5):
        got = _decode(dev, q, lens, pt, 30, 10.0, slopes, prefixes, n_splits)
        bu.assert_close(got, ref, z_max=Z, what=f"{n_splits}")


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("D,Hkv,G,start,n_new,ps,gs", [(64, 2, 8, 100, 70, 16, 16), (128, 2, 4, 0, 129, 64, 64),
                                                       (128, 1, 8, 777, 50, 32, 32), (256, 2, 8, 500, 33, 64, 64),
                                                       (256, 1, 4, 63, 200, 16, 16), (128, 3, 1, 40, 7, 64, 16),
                                                       (64, 1, 1, 5, 1, 16, 16)])
@pytest.mark.parametrize("shape", range(len(SHAPES)))
def test_chunks(kind, D, Hkv, G, start, n_new, ps, gs, shape):
    """Chunks in tiles of rows and as query windows; prefixes that end in the context, in the chunk,
    and behind it."""
    from int8_kv_cache_02_gb300 import binding
    n = start + n_new
    g, pt, dev, orc = _filled(kind, D + n_new, [n], Hkv, D, gs, ps)
    s = dict(SHAPES[shape])
    slopes = _slopes(Hkv * G) if s.pop("slopes", False) else None
    q = torch.randn((n_new, Hkv * G, D), generator=g).half()
    for prefix in ([4, start + n_new // 2, n + 100] if s.pop("prefixes", False) else [0]):
        ref = _reference(orc, q[None], [n], pt, s.get("window", 0), s.get("cap", 0.0), slopes,
                         [prefix])[0]
        for n_splits in (0, 1, 3, 40):
            got = _chunk(dev, q, start, pt[0], slopes=slopes, prefix=prefix, n_splits=n_splits, **s)
            bu.assert_close(got, ref, z_max=Z, what=f"prefix {prefix}, {n_splits} splits")
    assert binding.kv_pool_read_device_error(dev) == 0


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("size", [1.0, 30.0])
def test_scores_beyond_the_cap(kind, size):
    """Scores up to hundreds of caps: tanh near 1; caps so large that they change nothing, and the
    smallest."""
    lens, D, G = [400, 33], 128, 4
    g, pt, dev, orc = _filled(kind, 5, lens, 2, D, 32, 32, size)
    q = (size * torch.randn((2, 1, 2 * G, D), generator=g)).half()
    for cap in (0.5, 3.0, 8.0):
        ref = _reference(orc, q, lens, pt, cap=cap)
        # a score of x caps with a relative error e is off by e x (1 - tanh(x)^2) caps, at most
        # 0.45 e caps; e: the 16 roundings of a product's sum
        got = _decode(dev, q, lens, pt, cap=cap)
        bu.assert_close(got, ref, z_max=Z, what=f"cap {cap}")
        qc = q[:1].expand(60, 1, 2 * G, D).reshape(60, 2 * G, D).contiguous()
        bu.assert_close(_chunk(dev, qc, 340, pt[0], cap=cap),
                        _reference(orc, qc[None], [400], pt, cap=cap)[0], z_max=Z)
    if size == 1.0:
        for cap in (2.0 ** 64, 1e6):
            bu.assert_close(_decode(dev, q, lens, pt, cap=cap), _reference(orc, q, lens, pt), z_max=Z)
        got = _decode(dev, q, lens, pt, cap=2.0 ** -64)      # all weights alike
        mean = np.stack([orc.gather(0, pt[b].numpy(), n)[1].mean(axis=0) for b, n in enumerate(lens)])
        bu.assert_close(got[:, 0], mean.repeat(G, axis=1), z_max=Z)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("size", [60.0, 2000.0])
@pytest.mark.parametrize("D,Hkv,G", [(64, 1, 8), (128, 2, 4), (256, 1, 8)])
def test_large_scores(kind, size, D, Hkv, G):
    """Scores of 4e4 to 9e7 in base 2, windowed, with a prefix and (too small to be seen beside them)
    slopes: one position in the prefix wins by half its score, and the output is its V row; or all
    are alike, below a cap or beyond it, and it is the mean of the V rows that are seen."""
    lens, prefix, window, n_new = [700, 2500], 900, 300, 130
    g = torch.Generator().manual_seed(D)
    pt, n_pages = inputs.page_table(lens, 64, seed=D)
    sign = torch.where(torch.rand((Hkv, D), generator=g) < 0.5, -1.0, 1.0)
    q = (size * sign).repeat_interleave(G, 0).half().expand(n_new, Hkv * G, D).contiguous()
    for winner in (True, False):
        dev, orc = bu.make_pools(kind, Hkv, D, 16, 64, n_pages)
        for b, n in enumerate(lens):
            k = (sign * size).expand(1, n, Hkv, D).clone()
            if winner:
                k *= 0.5 * (torch.arange(n) % 2).view(1, n, 1, 1)
                k[:, n // 3] = sign * size
            v = torch.randn((1, n, Hkv, D), generator=g).half()
            bu.append(dev, orc, 0, k.half(), v, [0], pt[b:b + 1])
        caps = (0.0,) if winner else (0.0, 2.0 ** 30, 100.0)
        slopes = torch.full((Hkv * G,), 1e-6) if winner else None
        for cap in caps:
            q3 = q[None, :3].expand(2, 3, Hkv * G, D).contiguous()
            ref = _reference(orc, q3, lens, pt, window, cap, slopes, [prefix] * 2)
            for n_splits in (0, 1, 3):
                got = _decode(dev, q3, lens, pt, window, cap, slopes, [prefix] * 2, n_splits)
                bu.assert_close(got, ref, what=f"{winner} {cap} {n_splits}")
            for b, n in enumerate(lens):
                ref = _reference(orc, q[None], [n], pt[b:b + 1], window, cap, slopes, [prefix])[0]
                for n_splits in (0, 1, 3):
                    got = _chunk(dev, q, n - n_new, pt[b], window, cap, slopes, prefix, n_splits)
                    bu.assert_close(got, ref, what=f"chunk {winner} {cap} {n} {n_splits}")


@pytest.mark.parametrize("kind", KINDS)
def test_negative_scales_and_slopes(kind):
    """softmax_scale below 0; slopes of both signs and 0."""
    lens = [150, 31]
    g, pt, dev, orc = _filled(kind, 6, lens, 2, 64, 16, 16)
    q = torch.randn((2, 2, 8, 64), generator=g).half()
    slopes = torch.tensor([0.01, -0.01, 0.0, 0.5, 1.0, -0.02, 2.0, 0.1])
    ref = _reference(orc, q, lens, pt, 0, 3.0, slopes, scale=-0.2)
    bu.assert_close(_decode(dev, q, lens, pt, 0, 3.0, slopes, scale=-0.2), ref, z_max=Z)
    qc = q[:1].expand(64, 2, 8, 64).reshape(128, 8, 64).contiguous()
    ref = _reference(orc, qc[None], [150], pt, 0, 3.0, slopes, scale=-0.2)[0]
    bu.assert_close(_chunk(dev, qc, 22, pt[0], 0, 3.0, slopes, scale=-0.2), ref, z_max=Z)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("ps", [16, 32, 64, 128])
@pytest.mark.parametrize("window,prefix", [(100, 0), (100, 4), (33, 70), (1, 16), (500, 200)])
def test_pages_that_no_query_sees(kind, ps, window, prefix):
    """Entries between the prefix and the window that name no page: not looked at.  Rows behind the end
    hold NaN codes and scales."""
    from int8_kv_cache_02_gb300 import binding
    n, D, G = 1500, 128, 8
    g, pt, dev, orc = _filled(kind, 7, [n], 2, D, 16, ps)
    ref_table = pt.clone()
    end = int(pt[0, (n - 1) // ps])
    for t in (dev.k_store, dev.v_store):
        t.view(torch.uint8)[0, end, :, (n - 1) % ps + 1:] = 0x7F
    for t in (dev.k_scales, dev.v_scales):
        t[0, end, :, -(-((n - 1) % ps + 1) // 16):] = float("nan")
    for Q, chunk in ((1, False), (5, False), (40, True), (5, True)):
        q = torch.randn((1, Q, 2 * G, D), generator=g).half()
        first = n - Q + 1 - window                       # of the first query
        table = pt.clone()
        for lp in range(pt.shape[1]):
            if lp * ps >= prefix and (lp + 1) * ps <= first:
                table[0, lp] = -1
        ref = _reference(orc, q, [n], ref_table, window, 20.0, None, [prefix])
        for n_splits in (0, 1, 4):
            got = _chunk(dev, q[0], n - Q, table[0], window, 20.0, None, prefix, n_splits)[None] \
                if chunk else _decode(dev, q, [n], table, window, 20.0, None, [prefix], n_splits)
            bu.assert_close(got, ref, z_max=Z, what=f"{Q} {chunk} {n_splits}")
            assert binding.kv_pool_read_device_error(dev) == 0


@pytest.mark.parametrize("kind", KINDS)
def test_bad_pages_are_flagged_and_left_out(kind):
    from int8_kv_cache_02_gb300 import binding
    n, D, G, ps = 300, 64, 8, 16
    g, pt, dev, orc = _filled(kind, 8, [n], 1, D, 16, ps)
    pt[0, 3], pt[0, 9] = 10 ** 6, -1
    q = torch.randn((1, 64, G, D), generator=g).half()
    keep = np.array([p for p in range(n) if p // ps not in (3, 9)])
    kh, vh = (x[keep] for x in orc.gather(0, pt[0].clamp(0, 1).numpy(), n))
    for chunk in (False, True):
        got = _chunk(dev, q[0], n - 64, pt[0], cap=5.0)[None] if chunk else \
            _decode(dev, q, [n], pt, cap=5.0)
        assert binding.kv_pool_read_device_error(dev) == binding.DEVERR_PAGE_ID
        # (the positions left out lie before all queries)
        good, gt, gdev, gorc = _filled(kind, 8, [n], 1, D, 16, ps)
        kh, vh = (x[keep] for x in gorc.gather(0, gt[0].numpy(), n))
        ref = scored.attention(q[0].numpy(), kh, vh, len(keep), cap=5.0)[None]
        bu.assert_close(got, ref, z_max=Z, what=f"{chunk}")


@pytest.mark.parametrize("kind", KINDS)
def test_long_contexts(kind):
    """A window and a prefix at the far end of 60000 positions, in equal shares; slopes over the whole."""
    n, D, G = 60001, 64, 4
    g, pt, dev, orc = _filled(kind, 9, [n, 70], 1, D, 64, 64)
    q = torch.randn((2, 2, G, D), generator=g).half()
    slopes = _slopes(G)
    for window, prefixes in ((0, None), (4096, [5, 5]), (0, [60001, 3]), (20000, [30000, 1])):
        ref = _reference(orc, q, [n, 70], pt, window, 30.0, slopes, prefixes)
        bu.assert_close(_decode(dev, q, [n, 70], pt, window, 30.0, slopes, prefixes), ref, z_max=Z)
        if prefixes is None or prefixes[0] < n:
            qc = torch.randn((160, G, D), generator=g).half()
            p = prefixes[0] if prefixes else 0
            ref = _reference(orc, qc[None], [n], pt, window, 30.0, slopes, [p])[0]
            bu.assert_close(_chunk(dev, qc, n - 160, pt[0], window, 30.0, slopes, p), ref, z_max=Z)


def test_a_prefix_that_only_the_chunk_sees_and_replays():
    """Captured: lengths, prefixes and slopes are read on the device; on a stream of its own."""
    from int8_kv_cache_02_gb300 import binding
    D, H = 128, 8
    g, pt, dev, orc = _filled("e4m3", 10, [500, 500], 2, D, 32, 32)
    q, out = torch.randn((2, 1, H, D), generator=g).half(), torch.empty((2, H, D), device="cuda")
    lens, prefixes, slopes = _dev([1, 1]), _dev([0, 0]), torch.zeros(H, device="cuda")
    ws, dq, dpt = dev.decode_workspace(2, H, 8), q[:, 0].contiguous().cuda(), pt.cuda()
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(stream):
        with torch.cuda.graph(graph, stream=stream):
            binding.attn_decode_scored_int8(dev, 0, dq, lens, dpt, out, ws, window=40, softcap=9.0,
                                            slopes=slopes, prefix_lens=prefixes, n_splits=8)
        for n, p in (([500, 3], [10, 0]), ([0, 499], [3, 300]), ([77, 128], [0, 500])):
            s = torch.rand(H, generator=g) / 10
            for t, h in ((lens, torch.tensor(n)), (prefixes, torch.tensor(p)), (slopes, s)):
                t.copy_(h)
            graph.replay()
            stream.synchronize()
            bu.assert_close(out.cpu().numpy()[:, None], _reference(orc, q, n, pt, 40, 9.0, s, p),
                            z_max=Z)


@pytest.mark.parametrize("kind", KINDS)
def test_an_expired_wait_of_a_chunk_is_reported(kind):
    """As for plain chunks: the call completes, its rows count for nothing, and later ones are whole."""
    from int8_kv_cache_02_gb300 import binding as b
    n, G, D = 700, 8, 128
    g, pt, dev, orc = _filled(kind, 13, [n], 1, D, 64, 64)
    q = torch.randn((64, G, D), generator=g).half()
    args = (dev, q, n - 64, pt[0], 200, 9.0, _slopes(G), 70)
    for n_splits in (1, 3):
        want = _chunk(*args, n_splits)
        b.kv_pool_test_expire_prefill_waits(dev, 1000)
        got = _chunk(*args, n_splits)
        assert b.kv_pool_read_device_error(dev) == b.DEVERR_TIMEOUT and not got.any()
        b.kv_pool_test_expire_prefill_waits(dev, 0)
        assert np.array_equal(_chunk(*args, n_splits), want)


def test_two_streams_at_once():
    """Calls that share a pool and nothing else, on two streams: the bits of each alone."""
    from int8_kv_cache_02_gb300 import binding as b
    lens, D, H = [3000, 2999], 128, 8
    g, pt, dev, orc = _filled("int8", 14, lens, 2, D, 64, 64)
    q = torch.randn((2, 4, H, D), generator=g).half().cuda()
    alone = [_decode(dev, q.cpu(), lens, pt, 500, 20.0, _slopes(H), [7, 9], n_splits=n)
             for n in (5, 8)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    ws = [dev.decode_workspace(8, H, 8) for _ in range(2)]
    out = [torch.empty((2, 4, H, D), device="cuda") for _ in range(2)]
    dl, dpt, sl, pre = _dev(lens), pt.cuda(), _slopes(H).cuda(), _dev([7, 9])
    torch.cuda.synchronize()
    for _ in range(20):
        for k in range(2):
            b.attn_decode_scored_int8(dev, 0, q, dl, dpt, out[k], ws[k], window=500, softcap=20.0,
                                      slopes=sl, prefix_lens=pre, n_splits=(5, 8)[k],
                                      stream=streams[k])
    torch.cuda.synchronize()
    for k in range(2):
        assert np.array_equal(out[k].cpu().numpy(), alone[k])


def test_refusals():
    from int8_kv_cache_02_gb300 import binding as b
    g, pt, dev, orc = _filled("int8", 11, [64], 2, 64, 16, 16)
    q, out = (torch.zeros((1, 4, 64), dtype=t, device="cuda") for t in (torch.float16, torch.float32))
    call = lambda **kw: b.attn_decode_scored_int8(dev, 0, q, _dev([64]), pt.cuda(), out, None,  # noqa: E731
                                                  **{"n_splits": 1, **kw})
    chunk = lambda **kw: b.attn_prefill_chunk_scored_int8(dev, 0, q, 63, pt.cuda(), out, None,  # noqa: E731
                                                          **{"n_splits": 1, **kw})
    call(softcap=2.0 ** 64)
    for bad in (dict(softcap=-1.0), dict(softcap=float("nan")), dict(softcap=float("inf")),
                dict(softcap=2.0 ** -65), dict(softcap=2.0 ** 65), dict(window=-1),
                dict(n_splits=257), dict(softmax_scale=float("inf"))):
        for f in (call, chunk):
            with pytest.raises(b.Int8KVError, match="invalid"):
                f(**bad)
    with pytest.raises(b.Int8KVError, match="invalid"):
        chunk(prefix_len=-1)
    with pytest.raises(b.Int8KVError, match="workspace"):
        call(n_splits=4)
    for f in (call, chunk):
        with pytest.raises(TypeError):
            f(slopes=torch.zeros(4, dtype=torch.float16, device="cuda"))
        with pytest.raises(ValueError, match="slopes must have shape"):
            f(slopes=torch.zeros(3, device="cuda"))
    with pytest.raises(ValueError, match="prefix_lens must have shape"):
        call(prefix_lens=_dev([1, 2]))
    rows = b.KVPool(1, 2, 64, 64, 16, 4, "k8v8")
    for f in (b.attn_decode_scored_int8, b.attn_prefill_chunk_scored_int8):
        with pytest.raises(ValueError, match="block-scaled"):
            f(rows, 0, q, _dev([1]), pt.cuda(), out)
    assert b.lib().attn_decode_scored_int8(rows.handle, 0, q.data_ptr(), 1, 1, 4, pt.cuda().data_ptr(),
                                           pt.cuda().data_ptr(), 4, 0, 0.0, 0.0, None, None, 1,
                                           out.data_ptr(), None, 0, None) == -6


@pytest.mark.parametrize("kind", KINDS)
def test_a_speculative_step(kind):
    """As a server runs them: a prompt's chunk, then verify windows of ragged drafts: rotated append,
    window attention with capped scores, verification, and the refused tokens' pages back."""
    from int8_kv_cache_02_gb300 import binding as b
    S, n, H, Hkv, D, ps, V, cap = 3, 5, 8, 2, 128, 16, 300, 20.0
    g = torch.Generator().manual_seed(12)
    dev, orc = bu.make_pools(kind, Hkv, D, 16, ps, 64)
    tab = rope.table(400, D)
    dt = torch.from_numpy(tab).cuda()
    refs, table = _dev([0] * 64), torch.full((S, 16), -1, dtype=torch.int32, device="cuda")
    lens, pws = _dev([0] * S), dev.pages_workspace(S)
    prompt = [33, 7, 100]

    def rows(m):
        return tuple(torch.randn((S, m, h, D), generator=g).half() for h in (H, Hkv, Hkv))

    def oracle(q, k, v, pos, count):
        out = []
        for i in range(S):
            at = rope.rows_of(pos[i], count[i], R=D)
            rope.append(orc, 0, rope.turn(k[i, :count[i]].numpy(), tab, at, "halves"),
                        v[i, :count[i]].numpy(), pos[i], table[i].cpu().numpy())
            out.append(rope.turn(q[i, :count[i]].numpy(), tab, at, "halves").astype(np.float16))
        return out

    m = max(prompt)
    q, k, v = rows(m)
    out_q = torch.zeros((S, m, H, D), dtype=torch.float16, device="cuda")
    need = _dev(prompt)
    b.kv_pages_resize(dev, refs, table, need, pws)
    b.kv_rope_append(dev, 0, k.cuda(), v.cuda(), lens, table, dt, q=q.cuda(), q_out=out_q,
                     new_lens=need)
    want = oracle(q, k, v, [0] * S, prompt)
    lens.copy_(need)
    for i in range(S):
        out = torch.empty((prompt[i], H, D), device="cuda")
        b.attn_prefill_chunk_scored_int8(dev, 0, out_q[i, :prompt[i]].contiguous(), 0, table[i], out,
                                         softcap=cap, prefix_len=9, n_splits=1)
        kh, vh = orc.gather(0, table[i].cpu().numpy(), prompt[i])
        bu.assert_close(out.cpu().numpy(), scored.attention(want[i], kh, vh, prompt[i], cap=cap,
                                                            prefix=9), z_max=Z)
    at = list(prompt)
    for step in range(4):
        q, k, v = rows(n)
        out_q = torch.zeros((S, n, H, D), dtype=torch.float16, device="cuda")
        old = lens.clone()
        lens += n
        b.kv_pages_resize(dev, refs, table, lens, pws)
        b.kv_rope_append(dev, 0, k.cuda(), v.cuda(), old, table, dt, q=q.cuda(), q_out=out_q)
        want = oracle(q, k, v, at, [n] * S)
        out = torch.empty((S, n, H, D), device="cuda")
        ws = dev.decode_workspace(S * n, H, 8)
        b.attn_decode_scored_int8(dev, 0, out_q, lens, table, out, ws, softcap=cap, n_splits=8)
        ref = np.stack([scored.attention(want[i], *orc.gather(0, table[i].cpu().numpy(), at[i] + n),
                                         at[i] + n, cap=cap) for i in range(S)])
        bu.assert_close(out.cpu().numpy(), ref, z_max=Z)
        # the head of a model that is not here: logits by a fixed matrix
        logits = out.reshape(S, n, -1) @ torch.randn((H * D, V), generator=g).cuda()
        target = torch.softmax(logits, dim=2)
        draft = torch.softmax(logits[:, :n - 1] + 0.5, dim=2).roll(step % 2, 2).contiguous()
        x = target[:, :n - 1].argmax(dim=2).int()
        u, s = torch.rand((S, n - 1), generator=g), torch.rand((S,), generator=g)
        tokens, acc = torch.empty((S, n), dtype=torch.int32, device="cuda"), _dev([0] * S)
        b.kv_verify_drafts(target, x, u.cuda(), s.cuda(), tokens, acc, draft_probs=draft,
                           seq_lens=lens, seq_lens_out=lens)
        gone = verify.batch(target.cpu().numpy(), draft.cpu().numpy(), x.cpu().numpy(), u.numpy(),
                            s.numpy(), seq_lens=[a + n for a in at])
        assert np.array_equal(tokens.cpu().numpy(), gone[0]) and acc.tolist() == gone[1].tolist()
        assert lens.tolist() == gone[2].tolist()
        b.kv_pages_resize(dev, refs, table, lens, pws)
        at = lens.tolist()
        assert int(refs.sum()) == sum(math.ceil(a / ps) for a in at)
    assert b.kv_pool_read_device_error(dev) == 0


def _outliers(kind, n, D, seed, sign):
    """Keys [1][n][1][D], and the value that all of a query's dims have: every 16th key is the sign
    throughout (0: the two in turn), its score sign * value * D, and the others' scores are small
    beside it.  The value is a power of two and the codes are whole (e4m3: multiples of 2^-18 of their
    range), so that the sum of a row, and with it every score, is exact in fp32 whatever cancels in it."""
    g = torch.Generator().manual_seed(seed)
    size = 1024.0 if kind == "int8" else 128.0       # (e4m3 rounds codes to 2^-4, int8 to 1/254)
    k = 2 * torch.rand((1, n, 1, D), generator=g) - 1
    k[..., 0], k[..., 1] = 1.0, -1.0                 # (blocks of one scale)
    k -= k.mean(-1, keepdim=True)
    k = k.clamp(-1, 1)
    k[..., 0] = 1.0
    out = torch.arange(n) % 16 == seed % 16
    s = torch.ones(n) * sign if sign else 1.0 - 2.0 * (torch.arange(n) // 16 % 2)
    k[:, out] = s[out].view(1, -1, 1, 1)
    return k.half(), size


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("sign", [-1, 0])
def test_small_scores_beside_ones_beyond_the_cap(kind, D, sign):
    """One score in 16 is far beyond the cap, all negative or of both signs: those below -cap have no
    weight, and the others keep their precision beside them.  Chunk and decode of the same rows, against
    fp64."""
    n, G, n_new = 600, 8, 64
    k, size = _outliers(kind, n, D, 5, sign)
    g = torch.Generator().manual_seed(D)
    v = torch.randn((1, n, 1, D), generator=g).half()
    pt, n_pages = inputs.page_table([n], 64, seed=1)
    dev, orc = bu.make_pools(kind, 1, D, 64, 64, n_pages)
    bu.append(dev, orc, 0, k, v, [0], pt)
    q = torch.full((n_new, G, D), size).half()
    kh, _ = orc.gather(0, pt[0].numpy(), n)
    z = (kh.sum(-1)[:, 0] * size / math.sqrt(D)).astype(np.float64)
    out = np.arange(n) % 16 == 5
    far, near = np.abs(z[out]).min(), np.abs(z[~out]).max()
    scale = 10.0 / near / math.sqrt(D)             # small scores up to 10 (14.4 in base 2)
    for part in (1.3, 20.0, 500.0):                # the outliers in caps
        cap = float(far * 10.0 / near / part)
        assert cap > 0.5
        ref = _reference(orc, q[None], [n], pt, cap=cap, scale=scale)[0]
        for n_splits in (1, 3):
            got = _chunk(dev, q, n - n_new, pt[0], cap=cap, n_splits=n_splits, scale=scale)
            bu.assert_close(got, ref, z_max=Z, what=f"chunk, cap {cap}, {n_splits}")
        for Q in (1, 5, 64):
            got = _decode(dev, q[None, -Q:].contiguous(), [n], pt, cap=cap, scale=scale)[0]
            bu.assert_close(got, ref[-Q:], z_max=Z, what=f"decode of {Q}, cap {cap}")


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("D", [64, 256])
@pytest.mark.parametrize("slopes", [False, True])
@pytest.mark.parametrize("top", [10.0, 150.0])
def test_hidden_scores_change_no_bit(kind, D, slopes, top):
    """The keys of later tokens, or of ones that have left the window, are beyond the cap, or are not
    (with codes and scales of all others the same): the rows that do not see them have the same bits."""
    n, G, at, window = 300, 8, [40, 255, 299], 180
    k, size = _outliers(kind, n, D, 99, 1)
    k[:, 99 % 16::16] = k[:, :1]                    # (the outliers are set below)
    g = torch.Generator().manual_seed(D)
    v = torch.randn((1, n, 1, D), generator=g).half()
    q = torch.full((n, G, D), size).half()
    pt, n_pages = inputs.page_table([n], 64, seed=1)
    out, scale = [], None
    for big in (False, True):
        dev, orc = bu.make_pools(kind, 1, D, 16, 64, n_pages)
        kk = k.clone()
        if big:
            kk[:, at] = 1.0
        bu.append(dev, orc, 0, kk, v, [0], pt)
        z = np.abs(orc.gather(0, pt[0].numpy(), n)[0].sum(-1)[:, 0])
        if scale is None:
            scale = float(top / (z.max() * size))
        assert (z[at] * size * scale > 3 * top).all() if big else z.max() * size * scale < 1.1 * top
        out.append(_chunk(dev, q, 0, pt[0], window=window, cap=1.5 * top,
                          slopes=_slopes(G) if slopes else None, n_splits=1, scale=scale))
    P = np.arange(n)
    hidden = ~np.logical_or.reduce([(P >= a) & (P < a + window) for a in at])
    assert hidden[:40].all() and hidden[220:255].all() and hidden.sum() == 75
    assert np.array_equal(out[0][hidden], out[1][hidden])
    assert not np.array_equal(out[0][~hidden], out[1][~hidden])


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("prefix,cap", [(3500, 0.0), (9999, 20.0), (2111, 0.0)])
def test_biases_of_thousands_of_positions(kind, prefix, cap):
    """Queries thousands of positions ahead of a prefix's end, with slopes near 1 and of both signs: the
    biases are in the thousands where the weight is, and scores keep their precision beside them.  (A
    bias counted from the heaviest position is below 40 where a weight is above 2^-40, as above.)"""
    n, D, G = 3500, 64, 4
    g, pt, dev, orc = _filled(kind, 17, [n], 1, D, 64, 64)
    slopes = torch.tensor([0.84, 1.0, 0.2, -0.84])
    q = torch.randn((n, G, D), generator=g).half()
    ref = _reference(orc, q[None], [n], pt, 0, cap, slopes, [prefix])[0]
    for n_splits in (0, 1, 7):
        got = _chunk(dev, q, 0, pt[0], 0, cap, slopes, prefix, n_splits)
        bu.assert_close(got, ref, z_max=Z, what=f"{n_splits} splits")


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("D,G", [(64, 1), (128, 4), (256, 8)])
@pytest.mark.parametrize("window,prefix", [(0, 0), (0, 40), (3000, 0), (3000, 5), (900, 3200)])
def test_biases_that_grow_with_the_distance(kind, D, G, window, prefix):
    """Slopes below 0: the weight is at the first position that a query sees, thousands behind it; and
    above 0, with prefixes that a window does not reach."""
    lens = [4000, 3301, 17]
    g, pt, dev, orc = _filled(kind, 18, lens, 1, D, 32, 32)
    slopes = torch.tensor([-0.84, -1.0, 0.5, -0.03, 0.0, 1.0, -0.3, 2.0])[:G]
    for Q in (1, 3, 20):
        q = torch.randn((3, Q, G, D), generator=g).half()
        ref = _reference(orc, q, lens, pt, window, 30.0, slopes, [prefix] * 3)
        for n_splits in (0, 1, 3):
            got = _decode(dev, q, lens, pt, window, 30.0, slopes, [prefix] * 3, n_splits)
            bu.assert_close(got, ref, z_max=Z, what=f"{Q} queries, {n_splits} splits")
    n_new = 600 // G                    # (in tiles of rows)
    q = torch.randn((n_new, G, D), generator=g).half()
    for b in (0, 1):
        ref = _reference(orc, q[None], lens[b:b + 1], pt[b:b + 1], window, 0.0, slopes, [prefix])[0]
        got = _chunk(dev, q, lens[b] - n_new, pt[b], window, 0.0, slopes, prefix)
        bu.assert_close(got, ref, z_max=Z, what=f"chunk {b}")
