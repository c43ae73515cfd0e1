"""Block-scaled pools on the GPU: append bit for bit, attention against fp64."""

import numpy as np
import pytest
import torch

from int8_kv_cache_02_gb300 import inputs
from tests import block_util as bu

pytestmark = pytest.mark.gpu

KINDS = ["int8", "e4m3"]


def _rows(gen, n_seqs, n_new, Hkv, D, outliers=False):
    k = torch.randn((n_seqs, n_new, Hkv, D), generator=gen)
    if outliers:
        k[..., :4] *= 20
    return k.half(), torch.randn((n_seqs, n_new, Hkv, D), generator=gen).half()


# ---- append ----------------------------------------------------------------

@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("D,Hkv,gs,ps", [(64, 3, 16, 16), (64, 1, 16, 128), (128, 2, 64, 64),
                                         (256, 2, 32, 64), (256, 1, 128, 128), (128, 1, 16, 32)])
def test_append_is_bit_exact(kind, D, Hkv, gs, ps):
    """Prompts of ragged lengths, then single tokens, then a chunk behind an odd position."""
    g = torch.Generator().manual_seed(D + gs)
    lens = [1, gs - 1, 2 * gs + 3]
    room = [n + 3 * gs + 12 for n in lens]
    pt, n_pages = inputs.page_table(room, ps, seed=1)
    dev, orc = bu.make_pools(kind, Hkv, D, gs, ps, n_pages)
    for b, n in enumerate(lens):
        k, v = _rows(g, 1, n, Hkv, D, outliers=True)
        bu.append(dev, orc, 0, k, v, [0], pt[b:b + 1])
    bu.assert_same(dev, orc, "prompts")
    pos = list(lens)
    for step in range(6):         # magnitudes that rise make blocks grow, one of them steeply
        k, v = _rows(g, 3, 1, Hkv, D)
        k, v = (k * 2.0 ** step).half(), (v * 9.0 ** (step == 3)).half()
        bu.append(dev, orc, 0, k, v, pos, pt)
        pos = [p + 1 for p in pos]
        bu.assert_same(dev, orc, f"step {step}")
    k, v = _rows(g, 3, 3 * gs + 1, Hkv, D)
    bu.append(dev, orc, 0, (300 * k).half(), v, pos, pt)
    bu.assert_same(dev, orc, "chunk")


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("n_new", [1, 2, 5, 17, 64])
def test_append_sizes(kind, n_new):
    """Every launch shape of the kernel, in the second layer, at even and odd positions."""
    g = torch.Generator().manual_seed(n_new)
    pos = [0, 7, 64, 100]
    for D in (64, 128, 256):
        pt, n_pages = inputs.page_table([p + n_new for p in pos], 64, seed=2)
        dev, orc = bu.make_pools(kind, 2, D, 64, 64, n_pages, n_layers=2)
        for b, p in enumerate(pos):
            if p:
                bu.append(dev, orc, 1, *_rows(g, 1, p, 2, D), [0], pt[b:b + 1])
        bu.append(dev, orc, 1, *_rows(g, 4, n_new, 2, D, outliers=True), pos, pt)
        bu.assert_same(dev, orc, f"D {D}")


@pytest.mark.parametrize("kind", KINDS)
def test_append_rounds_ties_and_extremes_like_the_oracle(kind):
    """Quotients at and next to the codes' rounding boundaries; the largest and the smallest
    fp16 values; zeros."""
    D, gs = 256, 16
    q = 127.0 if kind == "int8" else 448.0
    if kind == "int8":
        y = np.arange(D) - 128 + 0.5                                  # half-integers
    else:
        t = np.sort(bu.oblock._POS)
        y = np.resize((t[1:] + t[:-1]) / 2, D)                        # midpoints of codes
    rows = []
    for s in (1.0, 0.25, 0.0078125):
        x = (y * s).astype(np.float16)
        x[0] = q * s                                                  # the scale is s exactly
        bits = x.view(np.int16)
        rows += [x, (bits + 1).view(np.float16), (bits - 1).view(np.float16)]
        rows[-1][0] = rows[-2][0] = q * s
    tiny = np.zeros(D, np.float16)
    tiny[:3] = [6e-8, -6e-8, 1.2e-7]
    rows += [tiny, np.full(D, 65504, np.float16), -np.full(D, 65504, np.float16),
             np.zeros(D, np.float16)]
    x = torch.tensor(np.stack(rows)).reshape(1, len(rows), 1, D)
    pt = torch.arange(len(rows), dtype=torch.int32).reshape(1, -1)
    dev, orc = bu.make_pools(kind, 1, D, gs, 16, len(rows))
    for i in range(len(rows)):                                        # a block for each row
        bu.append(dev, orc, 0, x[:, i:i + 1], x[:, i:i + 1].flip(3).contiguous(), [16 * i], pt)
    bu.assert_same(dev, orc)


@pytest.mark.parametrize("kind", KINDS)
def test_append_leaves_everything_else_alone(kind):
    from int8_kv_cache_02_gb300 import binding as b
    g = torch.Generator().manual_seed(3)
    dev, orc = bu.make_pools(kind, 2, 64, 16, 32, 6)
    for t in (dev.k_store, dev.v_store, orc.k_store, orc.v_store):
        (t.view(torch.uint8) if isinstance(t, torch.Tensor) else t.view(np.uint8))[...] = 0x35
    for t in (dev.k_scales, dev.v_scales, orc.k_scales, orc.v_scales):
        t[...] = 0.5
    pt = torch.tensor([[4, 1, -1], [0, 9, 2]], dtype=torch.int32)
    bu.append(dev, orc, 0, *_rows(g, 2, 20, 2, 64), [5, 0], pt)
    bu.assert_same(dev, orc)
    assert b.kv_pool_read_device_error(dev) == 0
    # a page that is not there, one beyond the pool, positions beyond the row and below 0
    bu.append(dev, orc, 0, *_rows(g, 2, 70, 2, 64), [40, 10], pt)
    bu.assert_same(dev, orc)
    assert b.kv_pool_read_device_error(dev) == b.DEVERR_PAGE_ID | b.DEVERR_LENGTH
    bu.append(dev, orc, 0, *_rows(g, 2, 4, 2, 64), [-2, 2 ** 31 - 2], pt)
    bu.assert_same(dev, orc)
    assert b.kv_pool_read_device_error(dev) == b.DEVERR_LENGTH


# ---- decode ----------------------------------------------------------------

def _filled(kind, seed, lens, Hkv, G, D, gs, ps, Q=1, outliers=False):
    g = torch.Generator().manual_seed(seed)
    pt, n_pages = inputs.page_table(lens, ps, seed=seed)
    dev, orc = bu.make_pools(kind, Hkv, D, gs, ps, n_pages)
    for b, n in enumerate(lens):
        if n:
            bu.append(dev, orc, 0, *_rows(g, 1, n, Hkv, D, outliers), [0], pt[b:b + 1])
    return torch.randn((len(lens), Q, Hkv * G, D), generator=g).half(), pt, dev, orc


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("D,Hkv,G,gs,ps", [(64, 2, 4, 16, 16), (64, 1, 8, 32, 128),
                                           (128, 2, 8, 64, 64), (128, 3, 1, 16, 32),
                                           (256, 2, 8, 64, 64), (256, 1, 3, 128, 128)])
def test_decode_against_fp64(kind, D, Hkv, G, gs, ps):
    from int8_kv_cache_02_gb300 import binding as b
    lens = [0, 1, 15, 16, 17, 63, 64, 65, 257, 700]
    q, pt, dev, orc = _filled(kind, D + G, lens, Hkv, G, D, gs, ps)
    ref = bu.reference(orc, 0, q, lens, pt)
    for n_splits in (0, 1, 2, 5, 33):
        out = bu.decode(dev, 0, q, lens, pt, n_splits=n_splits)
        bu.assert_close(out, ref, what=f"splits {n_splits}")
    assert b.kv_pool_read_device_error(dev) == 0


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("window", [1, 2, 16, 17, 100, 5000])
def test_decode_windows(kind, window):
    lens = [0, 1, 16, 130, 1003]
    q, pt, dev, orc = _filled(kind, window, lens, 2, 4, 128, 32, 64)
    ref = bu.reference(orc, 0, q, lens, pt, window)
    free = pt.clone()        # pages behind the window may be gone
    for b, n in enumerate(lens):
        free[b, :max(0, n - window) // 64] = -1
    for n_splits in (0, 1, 7):
        bu.assert_close(bu.decode(dev, 0, q, lens, free, window, n_splits), ref)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("D,Hkv,G,Q", [(64, 2, 4, 2), (128, 2, 3, 3), (128, 1, 8, 5),
                                       (256, 2, 8, 2), (64, 1, 1, 64), (256, 1, 5, 7),
                                       (128, 2, 1, 3), (128, 1, 8, 64)])
def test_query_windows(kind, D, Hkv, G, Q):
    lens = [0, 1, Q, 70, 403]        # queries at negative positions get zero rows
    q, pt, dev, orc = _filled(kind, D + Q, lens, Hkv, G, D, 16, 32, Q)
    ref = bu.reference(orc, 0, q, lens, pt)
    for n_splits in (0, 1, 2, 9):
        bu.assert_close(bu.decode(dev, 0, q, lens, pt, n_splits=n_splits), ref,
                        what=f"splits {n_splits}")


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("D,Hkv,G,Q,window", [(64, 1, 8, 1, 0), (64, 2, 2, 3, 0), (128, 2, 4, 1, 300),
                                              (128, 1, 4, 2, 0), (256, 1, 8, 1, 0),
                                              (256, 2, 3, 1, 700)])
def test_contexts_of_middling_length(kind, D, Hkv, G, Q, window):
    """A unit's tiles divided among a cluster's blocks (8 splits and more), some of which
    then have none, against fp64; fewer splits take the shares."""
    lens = [0, 1, 127, 129, 1300, 1999]
    q, pt, dev, orc = _filled(kind, D + window, lens, Hkv, G, D, 32, 64, Q)
    ref = bu.reference(orc, 0, q, lens, pt, window)
    outs = [bu.decode(dev, 0, q, lens, pt, window, n) for n in (0, 8, 64, 7, 1)]
    for out in outs:
        bu.assert_close(out, ref)
    assert np.array_equal(outs[0], outs[1]) and np.array_equal(outs[1], outs[2])


@pytest.mark.parametrize("kind", KINDS)
def test_layers_and_pages_behind_four_gigabytes(kind):
    """Two layers, the second one's pages at byte offsets past 2^32 in each store."""
    from int8_kv_cache_02_gb300 import binding as b
    Hkv, D, ps, n_pages, lens = 8, 128, 64, 40000, [130, 65]
    dev = b.KVPool(2, Hkv, D, 32, ps, n_pages, bu.KINDS[kind])
    assert dev.k_store.numel() > 2 ** 32
    pt = torch.tensor([[39999, 5, 39900], [39998, 39000, -1]], dtype=torch.int32)
    small = torch.tensor([[0, 1, 2], [3, 4, -1]], dtype=torch.int32)
    orc = bu.oblock.BlockPool(2, Hkv, D, 32, ps, 5, kind)
    g = torch.Generator().manual_seed(3)
    q = torch.randn((2, 1, 2 * Hkv, D), generator=g).half()
    for layer in (0, 1):
        for i, n in enumerate(lens):
            k, v = _rows(g, 1, n, Hkv, D)
            bu.append(dev, None, layer, k, v, [0], pt[i:i + 1])
            orc.append(layer, k.numpy(), v.numpy(), [0], small[i:i + 1].numpy())
    for layer in (0, 1):
        for n_splits in (1, 6):
            out = bu.decode(dev, layer, q, lens, pt, n_splits=n_splits)
            bu.assert_close(out, bu.reference(orc, layer, q, lens, small), what=f"layer {layer}")
    b.kv_pages_copy(dev, torch.tensor([39999, 39998], dtype=torch.int32, device="cuda"),
                    torch.tensor([7, 39997], dtype=torch.int32, device="cuda"))
    for x, y in ((39999, 7), (39998, 39997)):
        for t in (dev.k_store, dev.v_store):
            t = t.view(torch.uint8)
            assert t[1, x].any() and torch.equal(t[:, x], t[:, y])
    assert b.kv_pool_read_device_error(dev) == 0


@pytest.mark.parametrize("kind", KINDS)
def test_many_sequences(kind):
    """More sequences than the lanes that look for a share's place take in one step."""
    lens = [(7 * i) % 90 for i in range(700)]
    lens[300], lens[699] = 5000, 3001
    q, pt, dev, orc = _filled(kind, 21, lens, 1, 4, 64, 16, 16)
    ref = bu.reference(orc, 0, q, lens, pt)
    for n_splits in (0, 2, 4):
        bu.assert_close(bu.decode(dev, 0, q, lens, pt, n_splits=n_splits), ref)


@pytest.mark.parametrize("kind", KINDS)
def test_fused_append_behind_long_contexts(kind):
    """The decode kernel starts under its append: the last block of each sequence lies in the
    first, a middle and a late batch of a warp's tiles, and grows."""
    from int8_kv_cache_02_gb300 import binding as b
    for D, gs in ((64, 128), (128, 16), (256, 64)):
        lens = [1, 129, 3000, 9001]
        q, pt, dev, orc = _filled(kind, D, lens, 1, 4, D, gs, 128)
        g = torch.Generator().manual_seed(2)
        for n_splits in (1, 3, 40):
            k, v = _rows(g, 4, 1, 1, D)
            k = (4 * n_splits * k).half()
            pos = [n - 1 for n in lens]
            orc.append(0, k.numpy(), v.numpy(), pos, pt.numpy())
            out = torch.full((4, 4, D), float("nan"), device="cuda")
            ws = dev.decode_workspace(4, 4, n_splits)
            b.attn_decode_append_int8(dev, 0, q[:, 0].contiguous().cuda(),
                                      k[:, 0].contiguous().cuda(), v[:, 0].contiguous().cuda(),
                                      torch.tensor(lens, dtype=torch.int32, device="cuda"),
                                      pt.cuda(), out, ws, n_splits=n_splits)
            ref = bu.reference(orc, 0, q, lens, pt)[:, 0]
            bu.assert_close(out.cpu().numpy(), ref, z_max=600, what=f"{D} {n_splits}")
            bu.assert_same(dev, orc)


@pytest.mark.parametrize("kind", KINDS)
def test_decode_outliers_and_large_scores(kind):
    """Four K channels of 20 times the others' size: scores up to about 100 in base 2."""
    lens = [777, 64]
    q, pt, dev, orc = _filled(kind, 5, lens, 2, 8, 256, 64, 64, outliers=True)
    ref = bu.reference(orc, 0, q, lens, pt)
    bu.assert_close(bu.decode(dev, 0, q, lens, pt), ref, z_max=128)
    assert np.abs(bu.decode(dev, 0, q, lens, pt, scale=0.0) - ref).max() < 2e-3


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("rising", [True, False])
def test_decode_v_scales_of_any_range(kind, rising):
    """V magnitudes over 2^24 along the sequence, and a query that attends the small ones."""
    D, ps, n = 128, 16, 16 * 25
    g = torch.Generator().manual_seed(8)
    k, v = _rows(g, 1, n, 1, D)
    size = 2.0 ** -torch.arange(25).repeat_interleave(16).float()
    size = size.flip(0) if rising else size
    v = (v.float() * 64 * size[None, :, None, None]).half()
    small = size < 2.0 ** -12
    k[:, :, 0, 0] = torch.where(small, 9.0, -9.0).half()[None]
    q = torch.randn((1, 1, 4, D), generator=g).half()
    q[..., 0] = 24.0                         # scores of the small blocks win by 2^50
    pt, n_pages = inputs.page_table([n], ps, seed=8)
    dev, orc = bu.make_pools(kind, 1, D, 16, ps, n_pages)
    bu.append(dev, orc, 0, k, v, [0], pt)
    ref = bu.reference(orc, 0, q, [n], pt)
    for n_splits in (0, 1, 3):
        bu.assert_close(bu.decode(dev, 0, q, [n], pt, n_splits=n_splits), ref, z_max=64)


@pytest.mark.parametrize("kind", KINDS)
def test_decode_ignores_what_lies_behind_the_sequence(kind):
    """NaN codes, NaN and infinite scales in rows and blocks that are not attended."""
    lens = [37, 64, 5]
    q, pt, dev, orc = _filled(kind, 9, lens, 2, 4, 64, 16, 64)
    ref = bu.reference(orc, 0, q, lens, pt)
    for b, n in enumerate(lens):
        for t in (dev.k_store, dev.v_store):
            t.view(torch.uint8)[0, int(pt[b, 0]), :, n:] = 0x7F
        for t, x in ((dev.k_scales, float("nan")), (dev.v_scales, float("inf"))):
            t[0, int(pt[b, 0]), :, -(-n // 16):] = x
    for n_splits in (0, 1, 4):
        bu.assert_close(bu.decode(dev, 0, q, lens, pt, n_splits=n_splits), ref)


@pytest.mark.parametrize("kind", KINDS)
def test_zero_values_and_one_zero_block(kind):
    lens = [40]
    g = torch.Generator().manual_seed(10)
    k, v = _rows(g, 1, 40, 1, 64)
    v[:, :16] = 0
    k[:, 16:32] = 0
    pt, n_pages = inputs.page_table(lens, 16, seed=1)
    dev, orc = bu.make_pools(kind, 1, 64, 16, 16, n_pages)
    q = torch.randn((1, 1, 8, 64), generator=g).half()
    bu.append(dev, orc, 0, k, v, [0], pt)
    bu.assert_close(bu.decode(dev, 0, q, lens, pt), bu.reference(orc, 0, q, lens, pt))
    bu.append(dev, orc, 0, k, 0 * v, [0], pt)
    assert not bu.decode(dev, 0, q, lens, pt).any()


@pytest.mark.parametrize("kind", KINDS)
def test_bad_pages_and_lengths_are_flagged_and_left_out(kind):
    from int8_kv_cache_02_gb300 import binding as b
    lens = [64, 64]
    q, pt, dev, orc = _filled(kind, 11, lens, 1, 2, 64, 16, 32)
    bad = pt.clone()
    bad[0, 1], bad[1, 0] = -1, 10 ** 6
    out = bu.decode(dev, 0, q, lens, bad)
    assert b.kv_pool_read_device_error(dev) == b.DEVERR_PAGE_ID
    bu.assert_close(out[:1], bu.reference(orc, 0, q[:1], [32], pt))
    kh, vh = orc.gather(0, pt[1].numpy(), 64)
    bu.assert_close(out[1, 0], bu.oatt.decode(q[1, 0].numpy(), kh[32:], vh[32:], 32))
    out = bu.decode(dev, 0, q, [10 ** 9, -5], pt)
    assert b.kv_pool_read_device_error(dev) == b.DEVERR_LENGTH
    bu.assert_close(out[:1], bu.reference(orc, 0, q[:1], [64], pt))
    assert not out[1].any()


def test_long_ragged_batches_against_fp64_on_the_device():
    """Up to 40,000 positions: many shares per unit and many units per share."""
    from int8_kv_cache_02_gb300 import binding as b
    for kind, D, Hkv, G, lens in (("e4m3", 128, 4, 2, [40000, 3, 0, 12345, 1, 7777]),
                                  ("int8", 256, 1, 8, [33333]),
                                  ("int8", 64, 2, 5, [100] * 300 + [20000])):
        g = torch.Generator().manual_seed(len(lens))
        pt, n_pages = inputs.page_table(lens, 64, seed=4)
        dev, _ = bu.make_pools(kind, Hkv, D, 64, 64, n_pages)
        c = torch.randint(-127, 127, dev.k_store.shape, generator=g).to(torch.int8)
        if kind == "e4m3":
            c = c.view(torch.uint8).clamp(max=0x70).view(torch.int8)
        for t in (dev.k_store, dev.v_store):
            t.view(torch.int8).copy_(c)
            c = c.flip(3)
        m = 60.0 if kind == "int8" else 40.0
        dev.k_scales.copy_(torch.rand(dev.k_scales.shape, generator=g) / m)
        dev.v_scales.copy_(torch.rand(dev.v_scales.shape, generator=g) / m)
        q = torch.randn((len(lens), 1, Hkv * G, D), generator=g).half()
        out = torch.from_numpy(bu.decode(dev, 0, q, lens, pt))
        assert b.kv_pool_read_device_error(dev) == 0
        ref = torch.zeros(out.shape, dtype=torch.float64)
        for i, n in enumerate(lens):
            if n:
                ids = pt[i, :-(-n // 64)].long().cuda()
                x = []
                for t, s in ((dev.k_store, dev.k_scales), (dev.v_store, dev.v_scales)):
                    y = t.view(torch.uint8)[0][ids].view(t.dtype).float().double()
                    y = y * s[0][ids].double().repeat_interleave(64, 2)[..., None]
                    x.append(y.transpose(0, 1).reshape(Hkv, -1, D)[:, :n])
                z = q[i, 0].double().cuda().reshape(Hkv, G, D) @ x[0].transpose(1, 2) / D ** 0.5
                ref[i, 0] = (torch.softmax(z, -1) @ x[1]).reshape(-1, D).cpu()
        bu.assert_close(out.numpy(), ref.numpy(), z_max=64, what=kind)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("D,Hkv,G,start,n_new,ps", [
    (64, 2, 3, 0, 1, 16), (128, 2, 4, 0, 77, 64), (128, 1, 8, 1000, 130, 32), (256, 2, 8, 37, 20, 64),
    (256, 1, 1, 500, 65, 128), (64, 1, 5, 3, 300, 64)])
def test_prefill_chunk(kind, D, Hkv, G, start, n_new, ps):
    from int8_kv_cache_02_gb300 import binding as b
    n = start + n_new
    _, pt, dev, orc = _filled(kind, D + n_new, [n], Hkv, G, D, 16, ps)
    g = torch.Generator().manual_seed(n)
    q = torch.randn((n_new, Hkv * G, D), generator=g).half()
    kh, vh = orc.gather(0, pt[0].numpy(), n)
    ref = bu.oatt.prefill_chunk(q.numpy(), kh, vh, start)
    auto = b.attn_prefill_n_splits(dev, n_new, Hkv * G, start)
    for n_splits in (auto, 1, 2, 11):
        ws = torch.full((max(16, b.attn_prefill_workspace_bytes(n_new, Hkv * G, Hkv, D, n_splits)),),
                        255, dtype=torch.uint8, device="cuda")
        out = torch.full((n_new, Hkv * G, D), float("nan"), device="cuda")
        b.attn_prefill_chunk_int8(dev, 0, q.cuda(), start, pt[0].cuda(), out, ws,
                                  n_splits=0 if n_splits == auto else n_splits)
        bu.assert_close(out.cpu().numpy(), ref, what=f"splits {n_splits}")
    assert b.kv_pool_read_device_error(dev) == 0


def _one_winner(kind, D, Hkv, size, lens, ps, seed):
    """Pools whose sequences' position n // 3 beats the others by half its score: K rows there of
    +-size, and zeros or half as large elsewhere, beside queries of the same signs."""
    g = torch.Generator().manual_seed(seed)
    pt, n_pages = inputs.page_table(lens, ps, seed=seed)
    dev, orc = bu.make_pools(kind, Hkv, D, 16, ps, n_pages)
    sign = torch.where(torch.rand((Hkv, D), generator=g) < 0.5, -1.0, 1.0)
    for b, n in enumerate(lens):
        k, v = _rows(g, 1, n, Hkv, D)
        k = sign * size * 0.5 * (torch.arange(n) % 2).view(1, n, 1, 1)
        k[:, n // 3] = sign * size
        bu.append(dev, orc, 0, k.half(), v, [0], pt[b:b + 1])
    return sign, pt, dev, orc


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("size", [60.0, 2000.0])
@pytest.mark.parametrize("D,Hkv,G,Q", [(64, 2, 4, 1), (128, 1, 8, 1), (128, 2, 8, 2), (256, 2, 3, 1),
                                       (256, 1, 8, 3)])
def test_decode_of_large_scores(kind, size, D, Hkv, G, Q):
    """One position wins by far, with a score of 4e4 to 9e7 in base 2: the output is its V row.
    What is rounded are exponents relative to the winner's, so the bound is that of small
    scores; rounded at the scores' own size they would be off by 2^-9 and more."""
    lens = [1, 40, 700, 2500]
    sign, pt, dev, orc = _one_winner(kind, D, Hkv, size, lens, 64, D + G)
    q = (size * sign).repeat_interleave(G, 0).half().expand(len(lens), Q, Hkv * G, D).contiguous()
    ref = bu.reference(orc, 0, q, lens, pt)
    for n_splits in (0, 1, 3, 8):
        bu.assert_close(bu.decode(dev, 0, q, lens, pt, n_splits=n_splits), ref, what=f"{n_splits}")


def _prefill(dev, q, start, pt, n_splits=0, scale=0.0):
    """q [n_new][H][D] on the host -> fp32 of the same shape."""
    from int8_kv_cache_02_gb300 import binding as b
    n_new, H, D = q.shape
    ns = n_splits or b.attn_prefill_n_splits(dev, n_new, H, start)
    ws = torch.full((max(16, b.attn_prefill_workspace_bytes(n_new, H, dev.n_kv_heads, D, ns)),), 255,
                    dtype=torch.uint8, device="cuda")
    out = torch.full((n_new, H, D), float("nan"), device="cuda")
    b.attn_prefill_chunk_int8(dev, 0, q.cuda(), start, pt.cuda(), out, ws, softmax_scale=scale,
                              n_splits=n_splits)
    torch.cuda.synchronize()
    return out.cpu().numpy()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("D,Hkv,G,start,n_new,ps,gs,scale", [
    (64, 2, 8, 0, 64, 16, 16, 0.0),         # one whole tile of rows, positions in part
    (64, 1, 7, 130, 75, 32, 32, -0.1),      # rows of a query in two tiles, a negative scale
    (128, 2, 3, 63, 43, 16, 16, 0.0),       # a last tile of one row
    (128, 1, 1, 500, 128, 128, 128, 0.0),
    (256, 2, 5, 1, 26, 64, 32, 0.0),
    (256, 1, 8, 321, 17, 32, 16, -0.05)])
def test_prefill_in_tiles_of_rows(kind, D, Hkv, G, start, n_new, ps, gs, scale):
    """Rows, positions and splits that do not fill their tiles; NaN codes, NaN and infinite scales
    behind the chunk."""
    from int8_kv_cache_02_gb300 import binding as b
    n = start + n_new
    _, pt, dev, orc = _filled(kind, D + n_new, [n], Hkv, G, D, gs, ps)
    q = torch.randn((n_new, Hkv * G, D), generator=torch.Generator().manual_seed(n)).half()
    kh, vh = orc.gather(0, pt[0].numpy(), n)
    ref = bu.oatt.prefill_chunk(q.numpy(), kh, vh, start, scale or None)
    last = int(pt[0, (n - 1) // ps])
    for t in (dev.k_store, dev.v_store):
        t.view(torch.uint8)[0, last, :, (n - 1) % ps + 1:] = 0x7F
    for t, x in ((dev.k_scales, float("nan")), (dev.v_scales, float("inf"))):
        t[0, last, :, -(-((n - 1) % ps + 1) // gs):] = x
    for n_splits in (0, 1, 3, 40):          # (40: most blocks have no tile)
        bu.assert_close(_prefill(dev, q, start, pt[0], n_splits, scale), ref, z_max=16,
                        what=f"splits {n_splits}")
    assert b.kv_pool_read_device_error(dev) == 0


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("rising", [True, False])
def test_prefill_v_scales_of_any_range(kind, rising):
    """V magnitudes over 2^24 and zeros along the sequence; rows that attend the small ones."""
    D, ps, n, G = 128, 16, 16 * 26, 4
    g = torch.Generator().manual_seed(8)
    k, v = _rows(g, 1, n, 1, D)
    size = 2.0 ** -torch.arange(26).repeat_interleave(16).float()
    size[-16:] = 0
    size = size.flip(0) if rising else size
    v = (v.float() * 64 * size[None, :, None, None]).half()
    k[:, :, 0, 0] = torch.where(size < 2.0 ** -12, 9.0, -9.0).half()[None]
    pt, n_pages = inputs.page_table([n], ps, seed=8)
    dev, orc = bu.make_pools(kind, 1, D, 16, ps, n_pages)
    bu.append(dev, orc, 0, k, v, [0], pt)
    q = torch.randn((40, G, D), generator=g).half()
    q[..., 0] = 24.0
    kh, vh = orc.gather(0, pt[0].numpy(), n)
    ref = bu.oatt.prefill_chunk(q.numpy(), kh, vh, n - 40)
    for n_splits in (0, 1, 3):
        bu.assert_close(_prefill(dev, q, n - 40, pt[0], n_splits), ref, z_max=64)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("ps", [16, 64])
def test_prefill_flags_bad_pages_and_leaves_them_out(kind, ps):
    from int8_kv_cache_02_gb300 import binding as b
    n, n_new, G, D = 256, 32, 4, 128
    _, pt, dev, orc = _filled(kind, 3, [n], 1, G, D, 16, ps)
    q = torch.randn((n_new, G, D), generator=torch.Generator().manual_seed(1)).half()
    kh, vh = orc.gather(0, pt[0].numpy(), n)
    for lp, entry in ((0, -1), (64 // ps, 10 ** 6), (128 // ps, -(2 ** 31))):
        bad = pt.clone()
        bad[0, lp] = entry
        seen = np.arange(n) // ps != lp
        ref = bu.oatt.prefill_chunk(q.numpy(), kh[seen], vh[seen], n - n_new - ps)
        for n_splits in (1, 4):
            bu.assert_close(_prefill(dev, q, n - n_new, bad[0], n_splits), ref, what=f"{lp}")
            assert b.kv_pool_read_device_error(dev) == b.DEVERR_PAGE_ID
    gone = torch.full_like(pt, -1)          # no page at all: rows of zeros
    for n_splits in (1, 4):
        assert not _prefill(dev, q, n - n_new, gone[0], n_splits).any()
        assert b.kv_pool_read_device_error(dev) == b.DEVERR_PAGE_ID


@pytest.mark.parametrize("kind", KINDS)
def test_captured_prefill_chunks_with_one_workspace(kind):
    """Two captured chunks that share a workspace, replayed in turn with new queries; and a run
    on another stream gives the same bits."""
    from int8_kv_cache_02_gb300 import binding as b
    n, n_new, G, D = 700, 64, 4, 128
    _, pt, dev, orc = _filled(kind, 4, [n], 2, G, D, 64, 64)
    kh, vh = orc.gather(0, pt[0].numpy(), n)
    ptd = pt[0].cuda()
    q = [torch.zeros((n_new, 2 * G, D), dtype=torch.float16, device="cuda") for _ in range(2)]
    out = [torch.empty((n_new, 2 * G, D), device="cuda") for _ in range(2)]
    ws = torch.empty(b.attn_prefill_workspace_bytes(n_new, 2 * G, 2, D, 5), dtype=torch.uint8,
                     device="cuda")
    starts, graphs = (n - n_new, 100), []
    for i in range(2):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[i]):
            b.attn_prefill_chunk_int8(dev, 0, q[i], starts[i], ptd, out[i], ws, n_splits=5)
    g = torch.Generator().manual_seed(5)
    for _ in range(3):
        for i in range(2):
            q[i].copy_(torch.randn(q[i].shape, generator=g).half())
            graphs[i].replay()
        for i in range(2):
            ref = bu.oatt.prefill_chunk(q[i].cpu().numpy(), kh, vh, starts[i])
            bu.assert_close(out[i].cpu().numpy(), ref)
    other = torch.cuda.Stream()
    with torch.cuda.stream(other):
        again = _prefill(dev, q[0], starts[0], pt[0], 5)
    assert np.array_equal(again, out[0].cpu().numpy())


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("D,G,n_new,n", [(64, 8, 100, 500), (128, 4, 64, 500), (256, 8, 32, 500),
                                         (128, 4, 64, 6000)])
def test_an_expired_prefill_wait_is_reported_and_its_rows_count_for_nothing(kind, D, G, n_new, n):
    """The diagnostic withholds V: the wait for it gives up when weights and their sums are there
    already.  The error word tells, the rows are zeros, and the same pool gives the same bits as
    before once it is off."""
    from int8_kv_cache_02_gb300 import binding as b
    _, pt, dev, orc = _filled(kind, D, [n], 2, G, D, 32, 64)
    q = torch.randn((n_new, 2 * G, D), generator=torch.Generator().manual_seed(2)).half()
    for n_splits in (1, 3):
        want = _prefill(dev, q, n - n_new, pt[0], n_splits)
        assert b.kv_pool_read_device_error(dev) == 0 and want.any()
        b.kv_pool_test_expire_prefill_waits(dev, 1000)
        got = _prefill(dev, q, n - n_new, pt[0], n_splits)
        assert b.kv_pool_read_device_error(dev) == b.DEVERR_TIMEOUT
        assert not got.any(), n_splits
        b.kv_pool_test_expire_prefill_waits(dev, 0)
        assert np.array_equal(_prefill(dev, q, n - n_new, pt[0], n_splits), want)
        assert b.kv_pool_read_device_error(dev) == 0


def test_the_prefill_diagnostic_wants_a_block_scaled_pool_and_a_short_limit():
    from int8_kv_cache_02_gb300 import binding as b
    dev, _ = bu.make_pools("int8", 1, 64, 16, 16, 2)
    rows = b.KVPool(1, 1, 64, 64, 16, 2, "k8v8")
    for pool, us, status in ((rows, 10, "-6"), (dev, 1000001, "-1")):
        with pytest.raises(b.Int8KVError, match=status):
            b.kv_pool_test_expire_prefill_waits(pool, us)
    b.kv_pool_test_expire_prefill_waits(rows, 0)
    assert b.lib().kv_pool_test_expire_prefill_waits(None, 1) == -2


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("size", [60.0, 2000.0])
@pytest.mark.parametrize("D,Hkv,G,n_new", [(64, 1, 8, 64), (128, 2, 4, 40), (256, 1, 8, 20),
                                           (256, 2, 2, 10)])
def test_prefill_of_large_scores(kind, size, D, Hkv, G, n_new):
    """As for decode: one position before the chunk wins every row."""
    n = 700
    sign, pt, dev, orc = _one_winner(kind, D, Hkv, size, [n], 64, D + G)
    q = (size * sign).repeat_interleave(G, 0).half().expand(n_new, Hkv * G, D).contiguous()
    kh, vh = orc.gather(0, pt[0].numpy(), n)
    ref = bu.oatt.prefill_chunk(q.numpy(), kh, vh, n - n_new)
    for n_splits in (0, 1, 3):
        bu.assert_close(_prefill(dev, q, n - n_new, pt[0], n_splits), ref, what=f"{n_splits}")


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("size", [60.0, 2000.0])
@pytest.mark.parametrize("D,Hkv,G,Q", [(64, 2, 4, 1), (128, 1, 8, 1), (128, 2, 8, 2), (256, 2, 3, 1)])
def test_decode_of_large_equal_scores(kind, size, D, Hkv, G, Q):
    """All K rows alike: every score is the same, 4e4 to 9e7 in base 2, and the output the mean of
    the V rows, however many of them each partial has."""
    lens = [1, 40, 700, 2500]
    g = torch.Generator().manual_seed(D)
    pt, n_pages = inputs.page_table(lens, 64, seed=D)
    dev, orc = bu.make_pools(kind, Hkv, D, 16, 64, n_pages)
    sign = torch.where(torch.rand((Hkv, D), generator=g) < 0.5, -1.0, 1.0)
    for b, n in enumerate(lens):
        k = (size * sign).half().expand(1, n, Hkv, D).contiguous()
        bu.append(dev, orc, 0, k, 1 + _rows(g, 1, n, Hkv, D)[1], [0], pt[b:b + 1])
    q = (size * sign).repeat_interleave(G, 0).half().expand(len(lens), Q, Hkv * G, D).contiguous()
    ref = bu.reference(orc, 0, q, lens, pt)
    for n_splits in (0, 1, 3, 8, 40):
        bu.assert_close(bu.decode(dev, 0, q, lens, pt, n_splits=n_splits), ref, what=f"{n_splits}")


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("size", [60.0, 2000.0])
def test_prefill_of_large_equal_scores(kind, size):
    n, n_new, Hkv, G, D = 900, 70, 2, 3, 128
    g = torch.Generator().manual_seed(D)
    pt, n_pages = inputs.page_table([n], 64, seed=D)
    dev, orc = bu.make_pools(kind, Hkv, D, 16, 64, n_pages)
    sign = torch.where(torch.rand((Hkv, D), generator=g) < 0.5, -1.0, 1.0)
    k = (size * sign).half().expand(1, n, Hkv, D).contiguous()
    bu.append(dev, orc, 0, k, 1 + _rows(g, 1, n, Hkv, D)[1], [0], pt)
    q = (size * sign).repeat_interleave(G, 0).half().expand(n_new, Hkv * G, D).contiguous()
    kh, vh = orc.gather(0, pt[0].numpy(), n)
    ref = bu.oatt.prefill_chunk(q.numpy(), kh, vh, n - n_new)
    for n_splits in (0, 1, 2, 5):
        bu.assert_close(_prefill(dev, q, n - n_new, pt[0], n_splits), ref, what=f"{n_splits}")


def test_prefill_over_long_contexts():
    """The sums in tensor memory drop bits below their last place: an output takes n / 8 sums of
    products in a block (two parts of the weights for every 16 of its n positions), each of
    which loses at most 2^-23 of it."""
    n, n_new, D = 16384, 64, 128
    for kind, G in (("e4m3", 8), ("int8", 2)):
        dev, _ = bu.make_pools(kind, 1, D, 64, 64, n // 64)
        g = torch.Generator(device="cuda").manual_seed(1)
        pt = torch.randperm(n // 64, generator=g, device="cuda").int()[None]
        k, v = (torch.randn((1, n, 1, D), generator=g, device="cuda").half() for _ in range(2))
        from int8_kv_cache_02_gb300 import binding as b
        b.kv_quant_append(dev, 0, k, v, torch.zeros(1, dtype=torch.int32, device="cuda"), pt)
        q = torch.randn((n_new, G, D), generator=g, device="cuda").half()
        x = [(t.float().double() * s.double()[..., None]).reshape(-1, 64, D)[pt[0].long()].reshape(n, D)
             for t, s in ((dev.k_store, dev.k_scales.repeat_interleave(64, 3)),
                          (dev.v_store, dev.v_scales.repeat_interleave(64, 3)))]
        z = q.double() @ x[0].T / D ** 0.5                      # [n_new][G][n]
        at = torch.arange(n, device="cuda")
        z.masked_fill_((at > (n - n_new + torch.arange(n_new, device="cuda"))[:, None])[:, None],
                       float("-inf"))
        ref = torch.softmax(z, -1) @ x[1]
        for n_splits in (0, 1, 8):
            got = torch.from_numpy(_prefill(dev, q, n - n_new, pt[0], n_splits)).cuda()
            rel = ((got - ref).norm(dim=-1) / ref.norm(dim=-1)).max().item()
            block = n / (n_splits or b.attn_prefill_n_splits(dev, n_new, G, n - n_new))
            assert rel <= 2 * (6.6e-7 * 8 + 3 * 2.0 ** -21) + block / 8 * 2.0 ** -23, (kind, n_splits, rel)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("D,Hkv,G,n_new", [(64, 4, 8, 608), (128, 8, 4, 608), (256, 2, 8, 1216)])
def test_prefill_error_does_not_grow_with_the_context(kind, D, Hkv, G, n_new):
    """131,072 positions before a chunk whose blocks fill the device without splits, and the
    whole context in one block.  A sum in tensor memory is read out every 5120 positions, in which
    it takes 5120 / 8 sums of products that lose at most 2^-23 of it each."""
    from int8_kv_cache_02_gb300 import binding as b
    start = 131072
    n = start + n_new
    n_pages = -(-n // 64)
    dev, _ = bu.make_pools(kind, Hkv, D, 64, 64, n_pages)
    g = torch.Generator(device="cuda").manual_seed(1)
    pt = torch.randperm(n_pages, generator=g, device="cuda").int()[None]
    k, v = (torch.randn((1, n, Hkv, D), generator=g, device="cuda").half() for _ in range(2))
    b.kv_quant_append(dev, 0, k, v, torch.zeros(1, dtype=torch.int32, device="cuda"), pt)
    q = torch.randn((n_new, Hkv * G, D), generator=g, device="cuda").half()
    rows = torch.tensor([0, 1, n_new // 2, n_new - 2, n_new - 1], device="cuda")
    hide = torch.arange(n, device="cuda") > (start + rows)[:, None]
    ref = torch.empty((len(rows), Hkv, G, D), dtype=torch.float64, device="cuda")
    for h in range(Hkv):
        kh, vh = (t[0, :, h].float().double().mul_(s[0, :, h].double().repeat_interleave(64, 1)[..., None])
                  [pt[0].long()].reshape(-1, D)[:n]
                  for t, s in ((dev.k_store, dev.k_scales), (dev.v_store, dev.v_scales)))
        z = q[rows].double().view(-1, Hkv, G, D)[:, h] @ kh.T / D ** 0.5
        z.masked_fill_(hide[:, None], float("-inf"))
        ref[:, h] = torch.softmax(z, -1) @ vh
    ref = ref.reshape(len(rows), -1, D)
    for n_splits in (0, 1, 3):
        got = torch.from_numpy(_prefill(dev, q, start, pt[0], n_splits)).cuda()[rows]
        rel = ((got - ref).norm(dim=-1) / ref.norm(dim=-1)).max().item()
        assert rel <= 2 * (6.6e-7 * 8 + 3 * 2.0 ** -21) + 5120 / 8 * 2.0 ** -23, (n_splits, rel)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("levels", [(0, 4, 2), (3, 0, 5), (0, 66, 70), (0, 130, 300), (300, 80, 0)])
def test_prefill_sums_over_chains_whose_scores_move(kind, levels):
    """Three thirds of 5,440 positions whose scores differ by powers of two, with the V rows as far
    apart the other way: the sums that were read out are worth more, as much and nothing
    beside the next ones.  Rows in parts of a warp, of one block and of several splits."""
    n_new, G, D, third = 45, 3, 128, 5440
    n = 3 * third
    g = torch.Generator().manual_seed(sum(levels))
    k, v = _rows(g, 1, n, 1, D)
    level = torch.tensor(levels).repeat_interleave(third).float()
    k[:, :, 0, 0] = level * (D ** 0.5 / 24 / 1.4426950)
    v = (v.float() * torch.exp2(-level.clamp(max=8))[None, :, None, None]).half()
    pt, n_pages = inputs.page_table([n], 64, seed=8)
    dev, orc = bu.make_pools(kind, 1, D, 16, 64, n_pages)
    bu.append(dev, orc, 0, k, v, [0], pt)
    q = torch.randn((n_new, G, D), generator=g).half()
    q[..., 0] = 24.0
    kh, vh = orc.gather(0, pt[0].numpy(), n)
    ref = bu.oatt.prefill_chunk(q.numpy(), kh, vh, n - n_new)
    for n_splits in (1, 2, 3):
        out = _prefill(dev, q, n - n_new, pt[0], n_splits)
        assert np.array_equal(out, _prefill(dev, q, n - n_new, pt[0], n_splits))
        bu.assert_close(out, ref, z_max=max(levels) + 8 + 5120 / 8 * 2.0 ** -23 / (2 * 6.6e-7),
                        what=f"{n_splits}")


@pytest.mark.parametrize("kind", KINDS)
def test_prefill_of_more_units_than_the_device_has_places(kind):
    """2500 queries of 8/4 heads behind 70,000 positions: 40 tiles of rows for each of four kv
    heads, 160 blocks, so that some start when others end; pages of 16; and two splits."""
    from int8_kv_cache_02_gb300 import binding as b
    Hkv, G, D, n_new, start = 4, 2, 64, 2500, 70000
    n = start + n_new
    dev, _ = bu.make_pools(kind, Hkv, D, 16, 16, -(-n // 16))
    g = torch.Generator(device="cuda").manual_seed(1)
    pt = torch.randperm(-(-n // 16), generator=g, device="cuda").int()[None]
    k, v = (torch.randn((1, n, Hkv, D), generator=g, device="cuda").half() for _ in range(2))
    b.kv_quant_append(dev, 0, k, v, torch.zeros(1, dtype=torch.int32, device="cuda"), pt)
    q = torch.randn((n_new, Hkv * G, D), generator=g, device="cuda").half()
    rows = torch.tensor([0, 63, 64, 1250, 2495, 2499], device="cuda")
    hide = torch.arange(n, device="cuda") > (start + rows)[:, None]
    ref = torch.empty((len(rows), Hkv, G, D), dtype=torch.float64, device="cuda")
    for h in range(Hkv):
        kh, vh = ((t[0, :, h].float().double() * s[0, :, h].double().repeat_interleave(16, 1)[..., None])
                  [pt[0].long()].reshape(-1, D)[:n]
                  for t, s in ((dev.k_store, dev.k_scales), (dev.v_store, dev.v_scales)))
        z = q[rows].double().view(-1, Hkv, G, D)[:, h] @ kh.T / D ** 0.5
        z.masked_fill_(hide[:, None], float("-inf"))
        ref[:, h] = torch.softmax(z, -1) @ vh
    ref = ref.reshape(len(rows), -1, D)
    for n_splits in (0, 2):
        got = torch.from_numpy(_prefill(dev, q, start, pt[0], n_splits)).cuda()[rows]
        rel = ((got - ref).norm(dim=-1) / ref.norm(dim=-1)).max().item()
        assert rel <= 2 * (6.6e-7 * 8 + 3 * 2.0 ** -21) + 5120 / 8 * 2.0 ** -23, (n_splits, rel)


def test_long_chains_do_not_drift():
    """One block takes 32,768 positions alone: 512 tiles a warp.  The products' sums drop bits
    instead of rounding, so their error would grow with the chain (to 2e-5); sums rounded tile by
    tile keep the bound of assert_close."""
    from int8_kv_cache_02_gb300 import binding as b
    n, D = 32768, 128
    for kind, G in (("e4m3", 8), ("int8", 3)):
        dev, _ = bu.make_pools(kind, 1, D, 64, 64, n // 64)
        g = torch.Generator(device="cuda").manual_seed(1)
        pt = torch.arange(n // 64, dtype=torch.int32, device="cuda")[None]
        k, v = (torch.randn((1, n, 1, D), generator=g, device="cuda").half() for _ in range(2))
        b.kv_quant_append(dev, 0, k, v, torch.zeros(1, dtype=torch.int32, device="cuda"), pt)
        q = torch.randn((1, G, D), generator=g, device="cuda").half()
        x = [(t.float().double() * s.repeat_interleave(64, 3).double()[..., None]).reshape(n, D)
             for t, s in ((dev.k_store, dev.k_scales), (dev.v_store, dev.v_scales))]
        ref = torch.softmax(q[0].double() @ x[0].T / D ** 0.5, -1) @ x[1]
        lens = torch.tensor([n], dtype=torch.int32, device="cuda")
        for n_splits in (1, 2):
            out = torch.empty((1, G, D), device="cuda")
            b.attn_decode_int8(dev, 0, q, lens, pt, out, dev.decode_workspace(1, G, 2),
                               n_splits=n_splits)
            bu.assert_close(out[0].cpu().numpy(), ref.cpu().numpy(), what=f"{kind} {n_splits}")


# ---- calls together --------------------------------------------------------

@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("n_splits", [0, 1, 3])
def test_fused_append_is_append_then_decode(kind, n_splits):
    from int8_kv_cache_02_gb300 import binding as b
    lens = [0, 16, 100, 64]
    q, pt, dev, orc = _filled(kind, 12, [n + 1 for n in lens], 2, 4, 128, 16, 64)
    g = torch.Generator().manual_seed(1)
    k, v = _rows(g, 4, 1, 2, 128, outliers=True)
    n = torch.tensor([x + 1 for x in lens], dtype=torch.int32, device="cuda")
    out = torch.full((4, 8, 128), float("nan"), device="cuda")
    ws = dev.decode_workspace(4, 8, n_splits or 256)
    b.attn_decode_append_int8(dev, 0, q[:, 0].contiguous().cuda(), k[:, 0].contiguous().cuda(),
                              v[:, 0].contiguous().cuda(), n, pt.cuda(), out, ws,
                              n_splits=n_splits)
    orc.append(0, k.numpy(), v.numpy(), lens, pt.numpy())
    bu.assert_same(dev, orc)
    two = bu.decode(dev, 0, q, [x + 1 for x in lens], pt, n_splits=n_splits)
    assert np.array_equal(out.cpu().numpy(), two[:, 0])
    bu.assert_close(two, bu.reference(orc, 0, q, [x + 1 for x in lens], pt), z_max=64)


@pytest.mark.parametrize("kind", KINDS)
def test_captured_steps_replay_as_lengths_grow(kind):
    from int8_kv_cache_02_gb300 import binding as b
    B, H, Hkv, D, start, steps = 2, 8, 2, 128, [30, 61], 20
    g = torch.Generator().manual_seed(13)
    pt, n_pages = inputs.page_table([n + steps for n in start], 32, seed=3)
    dev, orc = bu.make_pools(kind, Hkv, D, 32, 32, n_pages)
    for i, n in enumerate(start):
        bu.append(dev, orc, 0, *_rows(g, 1, n, Hkv, D), [0], pt[i:i + 1])
    q = torch.zeros((B, H, D), dtype=torch.float16, device="cuda")
    k, v = (torch.zeros((B, Hkv, D), dtype=torch.float16, device="cuda") for _ in range(2))
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")       # empty while it is captured
    ptd, out = pt.cuda(), torch.empty((B, H, D), device="cuda")
    ws = dev.decode_workspace(B, H, 8)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b.attn_decode_append_int8(dev, 0, q, k, v, lens, ptd, out, ws, n_splits=8)
    for s in range(steps):
        ks, vs = _rows(g, B, 1, Hkv, D, outliers=s == 7)
        qs = torch.randn((B, 1, H, D), generator=g).half()
        q.copy_(qs[:, 0])
        k.copy_(ks[:, 0])
        v.copy_(vs[:, 0])
        pos = [n + s for n in start]
        lens.copy_(torch.tensor([p + 1 for p in pos], dtype=torch.int32))
        graph.replay()
        orc.append(0, ks.numpy(), vs.numpy(), pos, pt.numpy())
        ref = bu.reference(orc, 0, qs, [p + 1 for p in pos], pt)
        bu.assert_close(out.cpu().numpy(), ref[:, 0], z_max=64)
    bu.assert_same(dev, orc)
    assert b.kv_pool_read_device_error(dev) == 0


@pytest.mark.parametrize("kind", KINDS)
def test_results_do_not_depend_on_the_run_or_the_stream(kind):
    lens = [5000, 17, 900]
    q, pt, dev, orc = _filled(kind, 14, lens, 2, 4, 128, 64, 64)
    one = bu.decode(dev, 0, q, lens, pt)
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(other):
        two = bu.decode(dev, 0, q, lens, pt)
    assert np.array_equal(one, two)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("n_splits", [1, 3, 8])
def test_steps_read_what_the_kernels_just_before_them_wrote(kind, n_splits):
    """A captured step: lengths, tables and queries are written by the launches right before the
    fused call, whose decode starts under its append, and differ from replay to replay.  A row
    is on one set of pages in one replay and on the other, with other contents, in the next."""
    from int8_kv_cache_02_gb300 import binding as b
    lens = [700, 40, 1900, 129]
    q0, pt, dev, orc = _filled(kind, 31, [n + 8 for n in lens] * 2, 2, 4, 128, 16, 64)
    B, H, steps = len(lens), 8, 6
    g = torch.Generator().manual_seed(3)
    tables = torch.stack([pt[:B], pt[B:]])                       # [2][B][max_pages]
    qs = torch.randn((steps, B, 1, H, 128), generator=g).half()
    at = torch.tensor([[n + s // 2 + 1 for n in lens] for s in range(steps)], dtype=torch.int32)
    k, v = _rows(g, steps * B, 1, 2, 128)
    k, v = k.view(steps, B, 2, 128), v.view(steps, B, 2, 128)
    all_t, all_q, all_n, all_k, all_v = (x.cuda() for x in (tables, qs[:, :, 0].contiguous(), at, k, v))
    step = torch.zeros(1, dtype=torch.int64, device="cuda")
    table, q = torch.zeros_like(all_t[0]), torch.zeros_like(all_q[0])
    n, k1, v1 = torch.zeros_like(all_n[0]), torch.zeros_like(all_k[0]), torch.zeros_like(all_v[0])
    out, ws = torch.empty((B, H, 128), device="cuda"), dev.decode_workspace(B, H, n_splits)

    def run():
        for to, src, i in ((k1, all_k, step), (v1, all_v, step), (table, all_t, step % 2),
                           (n, all_n, step), (q, all_q, step)):
            torch.index_select(src, 0, i, out=to[None])
        b.attn_decode_append_int8(dev, 0, q, k1, v1, n, table, out, ws, n_splits=n_splits)
        step.add_(1)

    torch.index_select(all_q, 0, step, out=q[None])              # (loads its kernels)
    step % 2, step.add_(0)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    outs = []
    for s in range(steps):
        graph.replay()
        outs.append(out.clone())
    for s in range(steps):
        pos = (at[s] - 1).tolist()
        orc.append(0, k[s][:, None].numpy(), v[s][:, None].numpy(), pos, tables[s % 2].numpy())
        ref = bu.reference(orc, 0, qs[s], at[s].tolist(), tables[s % 2])
        bu.assert_close(outs[s].cpu().numpy(), ref[:, 0], what=f"step {s}")
    assert b.kv_pool_read_device_error(dev) == 0


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("n_splits,graph", [(1, False), (1, True), (3, True), (8, True)])
def test_forks_and_fused_steps_back_to_back(kind, n_splits, graph):
    """Nothing but the library's own launches, each of which may start under the one before it:
    row 2 becomes a fork of row 0, a step of all rows, a fork of row 1, a step, and so on. Each
    step's decode starts under its append and must see the table and lengths that the fork before
    that append wrote, not what the decode before them read."""
    from int8_kv_cache_02_gb300 import binding as b
    Hkv, G, D, ps, width, rows = 2, 4, 128, 64, 40, 3
    lens0 = [700, 2000]
    dev, orc = bu.make_pools(kind, Hkv, D, 32, ps, 120)
    refs = torch.zeros(120, dtype=torch.int32, device="cuda")
    table = torch.full((rows, width), -1, dtype=torch.int32, device="cuda")
    lens = torch.tensor(lens0 + [0], dtype=torch.int32, device="cuda")
    ws, dws = dev.pages_workspace(rows), dev.decode_workspace(rows, Hkv * G, n_splits)
    b.kv_pages_resize(dev, refs, table, lens, ws)
    g = torch.Generator().manual_seed(7)
    own = np.arange(rows * width).reshape(rows, width)
    for i, n in enumerate(lens0):
        k, v = _rows(g, 1, n, Hkv, D)
        bu.append(dev, None, 0, k, v, [0], table[i:i + 1].cpu())
        orc.append(0, k.numpy(), v.numpy(), [0], own[i:i + 1])
    steps = 10
    q = torch.randn((steps, rows, 1, Hkv * G, D), generator=g).half()
    k, v = (torch.randn((steps, rows, Hkv, D), generator=g).half() for _ in range(2))
    qd, kd, vd = q[:, :, 0].contiguous().cuda(), k.cuda(), v.cuda()
    out = torch.empty((steps, rows, Hkv * G, D), device="cuda")
    par = [torch.tensor([s % 2], dtype=torch.int32, device="cuda") for s in range(steps)]
    child = torch.tensor([2], dtype=torch.int32, device="cuda")

    def run():
        for s in range(steps):          # (a row's newest position is written again in each step)
            b.kv_pages_fork(dev, refs, table, lens, par[s], child, ws)
            b.attn_decode_append_int8(dev, 0, qd[s], kd[s], vd[s], lens, table, out[s], dws,
                                      n_splits=n_splits)

    if graph:
        cg = torch.cuda.CUDAGraph()
        with torch.cuda.graph(cg):
            run()
        cg.replay()
    else:
        run()
    torch.cuda.synchronize()
    n = list(lens0)
    for s in range(steps):
        p = s % 2
        for t in (orc.k_store, orc.v_store, orc.k_scales, orc.v_scales):
            t[0, own[2]] = t[0, own[p]]
        now = n + [n[p]]
        orc.append(0, k[s][:, None].numpy(), v[s][:, None].numpy(), [x - 1 for x in now], own)
        ref = bu.reference(orc, 0, q[s], now, torch.from_numpy(own))
        bu.assert_close(out[s].cpu().numpy(), ref[:, 0], what=f"step {s}")
    assert b.kv_pool_read_device_error(dev) == 0


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("window,gs,scale", [(1, 16, 0.0), (5, 64, -0.07), (16, 32, 0.0), (100, 128, 0.2),
                                             (3000, 16, -0.05)])
def test_fused_append_with_windows_and_scales(kind, window, gs, scale):
    """Windows that begin inside the block that the call appends to, and before it; negative
    softmax scales; rows of length 0 and 1."""
    from int8_kv_cache_02_gb300 import binding as b
    lens = [0, 1, 17, 128, 2000]
    q, pt, dev, orc = _filled(kind, window, lens, 2, 4, 128, gs, 128)
    g = torch.Generator().manual_seed(4)
    for n_splits in (1, 3, 8):
        k, v = _rows(g, 5, 1, 2, 128)
        pos = [n - 1 for n in lens]
        orc.append(0, k.numpy(), v.numpy(), pos, pt.numpy())
        out = torch.full((5, 8, 128), float("nan"), device="cuda")
        b.attn_decode_append_int8(dev, 0, q[:, 0].contiguous().cuda(), k[:, 0].contiguous().cuda(),
                                  v[:, 0].contiguous().cuda(),
                                  torch.tensor(lens, dtype=torch.int32, device="cuda"), pt.cuda(),
                                  out, dev.decode_workspace(5, 8, n_splits), window=window,
                                  softmax_scale=scale, n_splits=n_splits)
        ref = np.zeros(q.shape[:1] + q.shape[2:])
        for i, n in enumerate(lens):
            if n:
                kh, vh = orc.gather(0, pt[i].numpy(), n)
                ref[i] = bu.oatt.decode(q[i, 0].numpy(), kh, vh, n, window, scale or None)
        bu.assert_close(out.cpu().numpy(), ref, z_max=16, what=f"{n_splits}")
        bu.assert_same(dev, orc)


def test_noalloc_decode_and_refusals():
    import ctypes

    from int8_kv_cache_02_gb300 import binding as b
    lens = [900, 31]
    q, pt, dev, orc = _filled("int8", 15, lens, 2, 4, 128, 32, 64)
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    out = torch.empty((2, 8, 128), device="cuda")
    qd, ptd = q[:, 0].contiguous().cuda(), pt.cuda()
    b.attn_decode_int8_noalloc(dev, 0, qd, n, ptd, out)
    bu.assert_close(out.cpu().numpy(), bu.reference(orc, 0, q, lens, pt)[:, 0])
    status = lambda f: pytest.raises(b.Int8KVError, match=f)   # noqa: E731
    with status("-8"):
        b.attn_decode_int8(dev, 0, qd, n, ptd, out, None, n_splits=4)
    with status("-6"):
        b.kv_pool_set_decode_kernel(dev, b.DECODE_SIMT)
    with status("-6"):
        b.kv_pool_set_decode_kernel(dev, b.DECODE_WARP_MMA)
    b.kv_pool_set_decode_kernel(dev, b.DECODE_AUTO)
    with status("-5"):
        b.attn_prefill_chunk_int8(dev, 0, qd, 64 * pt.shape[1] - 1, ptd[0], out, n_splits=1)
    with status("-8"):
        b.attn_prefill_chunk_int8(dev, 0, qd, 900, ptd[0], out, n_splits=2)
    with pytest.raises(ValueError, match="one sequence"):
        b.attn_prefill_chunk_int8(dev, 0, qd, 0, ptd, out, n_splits=1)
    with status("-6"):
        b.kv_pool_save(dev, lens, ptd)
    with status("-6"):
        b.kv_pool_load(dev, b"I8KV" + bytes(60), ptd)
    with status("-6"):
        b.kv_pool_test_expire_waits(dev, 5)
    with status("-1"):
        b.attn_decode_int8(dev, 1, qd, n, ptd, out, None, n_splits=1)
    with status("-6"):
        b.attn_decode_int8(dev, 0, torch.zeros((2, 18, 128), dtype=torch.float16, device="cuda"),
                           n, ptd, torch.empty((2, 18, 128), device="cuda"), None, n_splits=1)
    assert b.lib().kv_quant_append(dev.handle, 0, ctypes.c_void_p(8), ctypes.c_void_p(16), 1, 1,
                                   ctypes.c_void_p(16), ctypes.c_void_p(16), 1, None) == -3
