"""Host-side checks of the block-scaled variants and the page calls (CPU only)."""

import ctypes

import pytest
import torch

from int8_kv_cache_02_gb300 import binding as b


@pytest.fixture(scope="module")
def L():
    from int8_kv_cache_02_gb300 import build
    build.build()
    return b.lib()


@pytest.mark.parametrize("variant", [b.K8V8_BLOCK, b.F8_BLOCK])
def test_region_bytes(L, variant):
    r = [b.int8kv_pool_region_bytes(2, 3, 128, 32, 64, 5, variant, k) for k in range(4)]
    rows = 2 * 5 * 3 * 64
    assert r == [rows * 128, rows * 128, rows // 32 * 4, rows // 32 * 4]


@pytest.mark.parametrize("args,status", [
    ((1, 2, 128, 64, 32, 1), -4),     # a block longer than a page
    ((1, 2, 128, 8, 64, 1), -4),      # not built
    ((1, 2, 128, 48, 64, 1), -4),
    ((1, 2, 128, 256, 128, 1), -4),
    ((1, 2, 96, 64, 64, 1), -6),
    ((1, 2, 128, 16, 48, 1), -6),
    ((1, 0, 128, 16, 64, 1), -1),
])
def test_refused_shapes(L, args, status):
    out = ctypes.c_size_t(0)
    for v in (b.K8V8_BLOCK, b.F8_BLOCK):
        assert L.int8kv_pool_region_bytes(*args, v, 0, ctypes.byref(out)) == status
        h, p = ctypes.c_void_p(), ctypes.c_void_p(0x10000)
        assert L.kv_pool_create(ctypes.byref(h), *args, v, p, p, p, p, None) == status


def test_create_refuses_missing_regions(L):
    h, p = ctypes.c_void_p(), ctypes.c_void_p(0x10000)
    odd = ctypes.c_void_p(0x10004)
    make = lambda *r: L.kv_pool_create(ctypes.byref(h), 1, 2, 64, 16, 16, 4,   # noqa: E731
                                       b.F8_BLOCK, *r, None)
    assert make(p, p, None, p) == -2 and make(p, p, p, None) == -2 and make(None, p, p, p) == -2
    assert make(p, p, odd, p) == -3


def test_page_calls_reject_null_pools(L):
    n = ctypes.c_size_t(0)
    assert L.kv_pages_workspace_bytes(None, 1, ctypes.byref(n)) == -2
    assert L.kv_pages_copy(None, 1, None, None, None) == -2
    assert L.kv_pages_resize(None, None, None, 1, 1, None, None, 0, None) == -2
    assert L.kv_pages_fork(None, None, None, 1, 1, None, 1, None, None, None, 0, None) == -2
    assert L.kv_pages_compact(None, None, None, 1, 1, None, None, None, None, 0, None) == -2


class _Pool:
    """Stand-in for a KVPool: the refusals below fire before its handle is used."""
    handle = None
    block, n_kv_heads, head_dim, n_pages = True, 2, 64, 4


def test_the_binding_refuses_host_tensors_and_shapes(L):
    i = torch.zeros(4, dtype=torch.int32)
    ws = torch.zeros(64, dtype=torch.uint8)
    for call in (lambda: b.kv_pages_copy(_Pool(), i, i),
                 lambda: b.kv_pages_resize(_Pool(), i, i.view(2, 2), i[:2], ws),
                 lambda: b.kv_pages_fork(_Pool(), i, i.view(2, 2), i[:2], i[:1], i[1:2], ws),
                 lambda: b.kv_pages_compact(_Pool(), i, i.view(2, 2), i, i.view(2, 2), i[:1], ws)):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    with pytest.raises(ValueError, match="shape"):
        b._shape(i, (3,), "i")
    k = torch.zeros((1, 1, 2, 128), dtype=torch.float16)
    with pytest.raises(ValueError, match="k_new must have shape"):
        b.kv_quant_append(_Pool(), 0, k, k, i[:1], i.view(1, 4))
    q = torch.zeros((1, 2, 32), dtype=torch.float16)
    with pytest.raises(ValueError, match="q must have shape"):
        b.attn_decode_int8(_Pool(), 0, q, i[:1], i.view(1, 4), q.float())
    q = torch.zeros((1, 2, 64), dtype=torch.float16)
    with pytest.raises(ValueError, match="seq_lens must have shape"):
        b.attn_decode_int8(_Pool(), 0, q, i, i.view(1, 4), q.float())
