"""Refusals of rotated appends and draft verification that need no GPU."""

import ctypes

import pytest
import torch

from int8_kv_cache_02_gb300 import binding as b


@pytest.fixture(scope="module")
def L():
    from int8_kv_cache_02_gb300 import build
    build.build()
    return b.lib()


P, ODD = 0x10000, 0x10008


def test_rope_append_rejects_a_null_pool(L):
    assert L.kv_rope_append(None, 0, None, None, None, 0, 0, 0, 1, 1, 1, None, None, None, 1, 64, 0,
                            None, 1, None, None, None, 1, None) == -2


class _Fake(ctypes.Structure):
    """The head of a pool's descriptor, which the refusals below look at before any CUDA call."""
    _fields_ = [(n, ctypes.c_int) for n in ("n_layers", "n_kv_heads", "head_dim", "group_size",
                                            "n_groups", "page_size", "n_pages", "variant")] + \
               [("rest", ctypes.c_ubyte * 1024)]


def _rope(L, **kw):
    a = dict(layer=0, q=P, k=P, v=P, qs=1024, ks=256, vs=256, n_seqs=2, n_new=3, n_heads=8, pos=P,
             lens=None, table=P, n_table=10, dim=64, style=0, positions=None, n_axes=1, axis=None,
             out=P, pages=P, max_pages=4)
    a.update(kw)
    f = _Fake(1, 2, 128, 128, 1, 64, 4, 0)
    status = L.kv_rope_append(ctypes.byref(f), *a.values(), None)
    words = [ctypes.addressof(x) if isinstance(x, ctypes.Array) else x or 0 for x in a.values()]
    assert L.kv_rope_append_packed(b._pack_rope(ctypes.addressof(f), *words, 0)) == status
    return status


@pytest.mark.parametrize("kw,status", [
    (dict(layer=1), -1), (dict(layer=-1), -1), (dict(n_seqs=-1), -1), (dict(n_new=-1), -1),
    (dict(max_pages=0), -1), (dict(n_table=0), -1), (dict(dim=0), -1), (dict(dim=24), -1),
    (dict(dim=144), -1), (dict(style=2), -1), (dict(n_axes=0), -1), (dict(n_axes=5), -1),
    (dict(n_heads=0), -1), (dict(qs=1023), -1), (dict(ks=255), -1), (dict(vs=0), -1),
    (dict(n_axes=2), -2), (dict(n_axes=2, axis=(ctypes.c_uint8 * 32)(*[2] * 32), positions=P), -1),
    (dict(n_axes=2, axis=(ctypes.c_uint8 * 32)(*[1] * 32)), -2),
    (dict(axis=(ctypes.c_uint8 * 32)(1)), -1),
    (dict(k=None), -2), (dict(v=None), -2), (dict(pos=None), -2), (dict(table=None), -2),
    (dict(pages=None), -2), (dict(out=None), -2),
    (dict(q=ODD), -3), (dict(k=ODD), -3), (dict(v=ODD), -3), (dict(out=ODD), -3),
    (dict(table=ODD), -3), (dict(qs=1028), -3), (dict(ks=260), -3), (dict(vs=260), -3),
    (dict(n_seqs=0), 0), (dict(n_new=0, k=None, v=None), 0),
])
def test_rope_append_refusals(L, kw, status):
    assert _rope(L, **kw) == status


def _verify(L, **kw):
    a = dict(batch=2, n_draft=3, vocab=100, target=P, ts=100, draft=P, ds=100, x=P, n=None, u=P, s=P,
             tokens=P, acc=P, lens=None, out=None)
    a.update(kw)
    status = L.kv_verify_drafts(*a.values(), None)
    assert L.kv_verify_drafts_packed(b._pack_verify(*(x or 0 for x in a.values()), 0)) == status
    return status


@pytest.mark.parametrize("kw,status", [
    (dict(batch=-1), -1), (dict(n_draft=-1), -1), (dict(vocab=0), -1), (dict(ts=99), -1),
    (dict(ds=99), -1), (dict(vocab=(1 << 30) + 1, ts=1 << 31, ds=1 << 31), -1),
    (dict(target=None), -2), (dict(x=None), -2), (dict(u=None), -2), (dict(s=None), -2),
    (dict(tokens=None), -2), (dict(acc=None), -2), (dict(lens=P), -2), (dict(out=P), -2),
    (dict(batch=1 << 28), -6), (dict(batch=0, target=None), 0),
])
def test_verify_refusals(L, kw, status):
    assert _verify(L, **kw) == status


@pytest.mark.parametrize("n", [(1 << 30) + 1, (1 << 31) - 256, (1 << 31) - 1])
def test_more_drafts_than_32_bits_count(L, n):
    """Indexes that step over 2^31 would never reach such a count.  (A batch of none: nothing runs.)"""
    assert _verify(L, batch=0, n_draft=n) == -1
    assert _verify(L, batch=0, n_draft=1 << 30) == 0


def test_packed_calls_refuse_null_and_read_floats(L):
    """The caps that are none are told by their value, so that a float's word is seen to arrive."""
    for f in (L.kv_rope_append_packed, L.kv_verify_drafts_packed, L.attn_decode_scored_int8_packed,
              L.attn_prefill_chunk_scored_int8_packed):
        assert f(None) == -2
    f = _Fake(1, 2, 128, 64, 1, 64, 4, 8)
    at = ctypes.addressof(f)
    for cap, status in ((1.0, 0), (-1.0, -1), (2.0 ** 65, -1), (float("nan"), -1), (0.0, 0)):
        words = b._pack_decode(at, 0, 0, 0, 1, 2, 0, 0, 4, 0, 0.0, cap, 0, 0, 1, 0, 0, 0, 0)
        assert L.attn_decode_scored_int8_packed(words) == status        # (a batch of none)
        words = b._pack_chunk(at, 0, 0, 0, 2, 0, 0, 4, 0, 0.0, cap, 0, 0, 1, 0, 0, 0, 0)
        assert L.attn_prefill_chunk_scored_int8_packed(words) == status
    words = b._pack_decode(at, 0, 0, 0, 1, 2, 0, 0, 4, 0, float("inf"), 1.0, 0, 0, 1, 0, 0, 0, 0)
    assert L.attn_decode_scored_int8_packed(words) == -1
    f.variant = 0
    words = b._pack_decode(at, 0, 0, 0, 1, 2, 0, 0, 4, 0, 0.0, 1.0, 0, 0, 1, 0, 0, 0, 0)
    assert L.attn_decode_scored_int8_packed(words) == -6        # not block-scaled


def test_packed_integers_beyond_32_bits_are_refused(L):
    """A window of 2^32 is not a window of 0: each integer in turn, one period of its type away from what
    the call would take (batches of none: nothing runs)."""
    f = _Fake(1, 2, 128, 64, 1, 64, 4, 8)
    at = ctypes.addressof(f)
    rope = [at, 0, 0, P, P, 1024, 256, 256, 0, 3, 8, P, 0, P, 10, 64, 0, 0, 1, 0, P, P, 4, 0]
    decode = [at, 0, 0, 0, 1, 2, 0, 0, 4, 0, 0.0, 1.0, 0, 0, 1, 0, 0, 0, 0]
    chunk = [at, 0, 0, 0, 2, 0, 0, 4, 0, 0.0, 1.0, 0, 0, 1, 0, 0, 0, 0]
    verify = [0, 3, 100, P, 100, 0, 0, P, 0, P, P, P, P, 0, 0, 0]
    for call, pack, words, ints in (
            (L.kv_rope_append_packed, b._pack_rope, rope, (1, 8, 9, 10, 14, 15, 16, 18, 22)),
            (L.attn_decode_scored_int8_packed, b._pack_decode, decode, (1, 3, 4, 5, 8, 9, 14)),
            (L.attn_prefill_chunk_scored_int8_packed, b._pack_chunk, chunk, (1, 3, 4, 5, 7, 8, 12, 13)),
            (L.kv_verify_drafts_packed, b._pack_verify, verify, (0, 1, 2))):
        assert call(pack(*words)) == 0
        for i in ints:
            for period in (1 << 32, -1 << 32, 5 << 32):
                off = list(words)
                off[i] += period
                assert call(pack(*off)) == -1, (call.__name__, i, period)


class _Pool:
    handle = None
    block, n_kv_heads, head_dim, n_pages, device_index = True, 2, 64, 4, 0


def test_the_binding_refuses(L):
    i, f = torch.zeros(4, dtype=torch.int32), torch.zeros(4)
    k = torch.zeros((1, 4, 2, 64), dtype=torch.float16)
    with pytest.raises(ValueError, match="k_new must have shape"):
        b.kv_rope_append(_Pool(), 0, k[0], k[0], i[:1], i.view(1, 4), f.view(1, 4))
    with pytest.raises(ValueError, match="CUDA"):
        b.kv_rope_append(_Pool(), 0, k, k, i[:1], i.view(1, 4), f.view(1, 4))
    with pytest.raises(ValueError, match="CUDA"):
        b.kv_verify_drafts(f.view(1, 2, 2), i[:1].view(1, 1), f[:1].view(1, 1), f[:1],
                           i[:2].view(1, 2), i[:1])


def test_token_and_row_strides():
    """What counts as evenly apart (on the host's device, -1; addresses are not looked at here)."""
    def tokens(t, heads=2, device=-1):
        return b._token_rows(t, (*t.shape[:2], heads, 64), device, "k")[1]

    def rows(t, *shape, device=-1):
        return b._prob_rows(t, shape, device, "p")[1]
    wide = torch.zeros((3, 5, 12, 64), dtype=torch.float16)
    assert tokens(wide[:, :, 2:4]) == 12 * 64
    assert tokens(wide[:, :1, :2]) == 5 * 12 * 64
    assert tokens(wide[:1, 1:4, :2]) == 12 * 64
    assert tokens(wide[:1, :1, :2]) == 128
    assert tokens(wide, 12) == 12 * 64 and tokens(wide[:, :0, :2]) == 128
    for t in (wide[:, :3, :2], wide.transpose(0, 1)[:, :, :2], wide[:, :, ::2][:, :, :2]):
        with pytest.raises(ValueError, match="evenly"):
            tokens(t)
    p = torch.zeros((2, 4, 40))
    assert rows(p[..., :33], 2, 4, 33) == 40 and rows(p[:, :1, :33], 2, 1, 33) == 160
    assert rows(p, 2, 4, 40) == 40 and rows(p[:, :0], 2, 0, 40) == 40
    with pytest.raises(ValueError, match="evenly"):
        rows(p[:, :3], 2, 3, 40)
    for call in (lambda: tokens(wide, device=0), lambda: rows(p, 2, 4, 40, device=0)):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    for call in (lambda: b._token_rows(None, (1, 1, 1, 64), 0, "k"),
                 lambda: b._prob_rows([1.0], (1, 1, 1), 0, "p"),
                 lambda: b._ptr(3, torch.int32, (1,), 0, "n")):
        with pytest.raises(TypeError, match="torch tensor"):
            call()


def test_one_test_where_all_is_well():
    i = torch.zeros((2, 6), dtype=torch.int32)
    assert b._ptr(i, torch.int32, (2, 6), -1, "i") == i.data_ptr()
    for t, dtype in ((i, torch.float32), (i[:, ::2], torch.int32), (i, torch.int32)):
        with pytest.raises(ValueError, match="i must be on a CUDA device"):
            b._ptr(t, dtype, (3, 6) if t is i else (2, 3), -1, "i")
