"""Oracle: rotated appends (test infrastructure only).

Pair i of the first R values of a row, (a, b) = values (i, i + R/2) ("halves") or (2i, 2i + 1)
("pairs"), with c and s from row ``position(axis of i)`` of the table:

    a' = fl(fl(a c) - fl(b s)),   b' = fl(fl(b c) + fl(a s))        in fp32

A position outside the table leaves its pairs as they are.  ``turn64`` is the same as complex
multiplication in fp64, written apart from it.
"""

import numpy as np

from . import q4
from .block import BlockPool


def table(n, R, base=10000.0):
    """fp32 [n][R]: cosines of the R / 2 pairs, then their sines; angles in fp64."""
    angle = np.arange(n)[:, None] * base ** (-np.arange(R // 2) / (R // 2))
    return np.concatenate([np.cos(angle), np.sin(angle)], axis=1).astype(np.float32)


def _pairs(R, style):
    i = np.arange(R // 2)
    return (i, i + R // 2) if style == "halves" else (2 * i, 2 * i + 1)


def turn(x16, tab, at, style):
    """x16: fp16 [T][heads][D]; at: int [T][R / 2], the table's row of each pair -> fp32."""
    x = np.asarray(x16, np.float16).astype(np.float32)
    R = tab.shape[1]
    i = np.arange(R // 2)
    ok = (at >= 0) & (at < tab.shape[0])
    row = np.where(ok, at, 0)
    c = np.where(ok, tab[row, i], np.float32(1))[:, None]
    s = np.where(ok, tab[row, R // 2 + i], np.float32(0))[:, None]
    ia, ib = _pairs(R, style)
    out = x.copy()
    a, b = x[..., ia], x[..., ib]
    out[..., ia] = a * c - b * s
    out[..., ib] = b * c + a * s
    return out


def turn64(x16, tab, at, style):
    x = np.asarray(x16, np.float16).astype(np.float64)
    R = tab.shape[1]
    i = np.arange(R // 2)
    e = tab[at, i].astype(np.float64) + 1j * tab[at, R // 2 + i].astype(np.float64)
    ia, ib = _pairs(R, style)
    z = (x[..., ia] + 1j * x[..., ib]) * e[:, None]
    out = x.copy()
    out[..., ia], out[..., ib] = z.real, z.imag
    return out


def rows_of(pos, n, positions=None, pair_axis=None, R=None):
    """The table's row of each (token, pair) of one sequence: int [n][R / 2].  positions: int
    [axes][n], or None: pos + i."""
    axis = np.zeros(R // 2, int) if pair_axis is None else np.asarray(pair_axis, int)
    p = (pos + np.arange(n))[None] if positions is None else np.asarray(positions)
    return p[axis].T


def append(orc, layer, k32, v16, pos, page_row):
    """K rows (fp32, turned) and V rows (fp16) [n][Hkv][D] of one sequence behind pos positions, into
    an oracle's pool of either kind.  Tokens without a place are left out."""
    if isinstance(orc, BlockPool):
        _append_blocks(orc, layer, k32, v16, pos, page_row)
    else:
        _append_rows(orc, layer, k32, v16, pos, page_row)


def _append_blocks(orc, layer, k32, v16, pos, page_row):
    gs, ps = orc.gs, orc.page_size
    for new, store, scales in ((k32, orc.k_store, orc.k_scales),
                               (v16.astype(np.float32), orc.v_store, orc.v_scales)):
        i = max(0, -pos)
        while i < len(new):
            at = pos + i
            n = min(gs - at % gs, len(new) - i)
            page = int(page_row[at // ps]) if at // ps < len(page_row) else -1
            if 0 <= page < orc.n_pages:
                for h in range(orc.n_kv_heads):
                    orc._block(store[layer, page, h], scales[layer, page, h], at % ps,
                               new[i:i + n, h])
            i += n


def _append_rows(orc, layer, k32, v16, pos, page_row):
    ps = orc.page_size
    for i in range(len(k32)):
        at = pos + i
        page = int(page_row[at // ps]) if 0 <= at // ps < len(page_row) else -1
        if not 0 <= page < orc.n_pages:
            continue
        for x, store, scales, is8, is4 in (
                (k32[i], orc.k_store, orc.k_scales, orc.k_int8, orc.k_q4),
                (v16[i].astype(np.float32), orc.v_store, orc.v_scales, orc.v_int8, orc.v_q4)):
            if is4:
                codes, d = q4.q4_0_quantize(q4.fwht(x))
                store[layer, page, :, at % ps, :] = q4.pack(codes)
                scales[layer, page, :, at % ps, :] = d
            elif is8:
                g = x.reshape(len(x), -1, orc.gs)
                s = (np.abs(g).max(axis=2) / np.float32(127)).astype(np.float16)
                f = s.astype(np.float32)[..., None]
                with np.errstate(divide="ignore", invalid="ignore"):
                    c = np.where(f == 0, np.float32(0), np.rint(g / f))
                store[layer, page, :, at % ps, :] = np.clip(c, -127, 127).reshape(x.shape)
                scales[layer, page, :, at % ps, :] = s
            else:
                store[layer, page, :, at % ps, :] = x.astype(np.float16)
