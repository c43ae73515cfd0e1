"""Helpers for the tests of block-scaled pools: fill a device pool and the oracle's from
the same fp16 inputs, compare them, and bound the attention's rounding errors."""

import numpy as np
import torch

from oracle import attention as oatt
from oracle import block as oblock

KINDS = {"int8": "k8v8_block", "e4m3": "f8_block"}


def make_pools(kind, Hkv, D, gs, ps, n_pages, n_layers=1):
    from int8_kv_cache_02_gb300 import binding, build
    build.build()
    dev = binding.KVPool(n_layers, Hkv, D, gs, ps, n_pages, KINDS[kind])
    return dev, oblock.BlockPool(n_layers, Hkv, D, gs, ps, n_pages, kind)


def append(dev, orc, layer, k, v, pos, pt):
    """k, v fp16 [n_seqs][n_new][Hkv][D] on the host, behind pos[b] positions, on both pools."""
    from int8_kv_cache_02_gb300 import binding
    binding.kv_quant_append(dev, layer, k.cuda(), v.cuda(),
                            torch.tensor(pos, dtype=torch.int32, device="cuda"), pt.cuda())
    if orc is not None:
        orc.append(layer, k.numpy(), v.numpy(), pos, pt.numpy())


def assert_same(dev, orc, what=""):
    """Every byte of the two pools is the same (e4m3: -0 and 0 count as one code)."""
    torch.cuda.synchronize()
    for name in ("k_store", "v_store", "k_scales", "v_scales"):
        d, o = getattr(dev, name), getattr(orc, name)
        d = d.view(torch.uint8).cpu().numpy().view(o.dtype) if "store" in name else d.cpu().numpy()
        if o.dtype == np.uint8:
            d, o = np.where(d == 0x80, 0, d), np.where(o == 0x80, 0, o)
        if not np.array_equal(d, o):
            bad = np.argwhere(d != o)
            at = tuple(bad[0])
            raise AssertionError(f"{what} {name}: {len(bad)} differ, first {at}: {d[at]} {o[at]}")


def reference(orc, layer, q, lens, pt, window=0):
    """fp64 [B][Q][H][D] of queries [B][Q][H][D], causal within the window of Q queries."""
    q = q.numpy()
    out = np.zeros(q.shape, np.float64)
    for b, n in enumerate(lens):
        n = max(int(n), 0)
        if n == 0:
            continue
        kh, vh = orc.gather(layer, pt[b].numpy(), n)
        for i in range(q.shape[1]):
            last = n - q.shape[1] + i + 1
            if last > 0:
                out[b, i] = oatt.decode(q[b, i], kh, vh, last, window)
    return out


def assert_close(out, ref, z_max=8.0, what=""):
    """fp32 attention outputs against fp64 ones.

    A score z (base 2, |z| <= z_max) is a sum of up to 256 exact products in fp32: about
    16 roundings' worth (their square root) of half a step 2^-24 |z| each, so a weight is off by
    ln 2 * 16 * 2^-24 * z_max = 6.6e-7 z_max, relative; the exponential and the weight's fp16 pair
    add 2^-21, the sums of the values as much.  An output is a weighted mean: the relative
    2-norm per head stays within that sum, taken twice for margin where errors add up."""
    tol = 2 * (6.6e-7 * z_max + 3 * 2.0 ** -21)
    out, ref = np.asarray(out, np.float64), np.asarray(ref)
    assert np.isfinite(out).all(), what
    nd = np.linalg.norm((out - ref).reshape(-1, out.shape[-1]), axis=1)
    nr = np.linalg.norm(ref.reshape(-1, out.shape[-1]), axis=1)
    assert np.all(nd[nr == 0] == 0), f"{what}: nonzero rows where nothing is attended"
    rel = float((nd[nr > 0] / nr[nr > 0]).max()) if (nr > 0).any() else 0.0
    assert rel <= tol, f"{what}: relative 2-norm {rel:.2e} > {tol:.2e}"
    return rel


def decode(dev, layer, q, lens, pt, window=0, n_splits=0, scale=0.0):
    """q [B][Q][H][D] on the host -> fp32 [B][Q][H][D]."""
    from int8_kv_cache_02_gb300 import binding
    B, Q, H, D = q.shape
    ws = dev.decode_workspace(B * Q, H, n_splits or 256)
    ws.fill_(0xFF)          # any contents will do
    out = torch.full((B, Q, H, D), float("nan"), dtype=torch.float32, device="cuda")
    lens = torch.tensor(lens, dtype=torch.int32, device="cuda")
    if Q == 1:
        binding.attn_decode_int8(dev, layer, q[:, 0].contiguous().cuda(), lens, pt.cuda(),
                                 out[:, 0].view(B, H, D), ws, window=window,
                                 softmax_scale=scale, n_splits=n_splits)
    else:
        binding.attn_decode_multi_int8(dev, layer, q.cuda(), lens, pt.cuda(), out, ws,
                                       softmax_scale=scale, n_splits=n_splits)
    torch.cuda.synchronize()
    return out.cpu().numpy()
