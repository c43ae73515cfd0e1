"""Oracle: the block-scaled 8-bit KV pool (test infrastructure only).

Every block of ``gs`` consecutive positions of one kv head has one fp32 scale s for
all its codes; value = code * s.  Codes are int8 (qmax 127) or e4m3 (qmax 448).
Appending new rows x of a block, with a = max |x|:

  the block's first position is new, or its scale is 0:  s = fp32(a / qmax)
  else  s = s_old * 2^k, the smallest k >= 0 with a <= fp32(fits * s_old) * 2^k,
        fits = 127.5 (int8) or 464 (e4m3); the older codes become round(c * 2^-k)
  new codes  round(fp32(x / s)), half to even, saturated at +-qmax; 0 where s = 0

e4m3: sign, 4 exponent bits (bias 7), 3 mantissa bits; exponent 0 is subnormal
(m / 8 * 2^-6); the code 0x7f is NaN, so the largest value is 448.
"""

import numpy as np

QMAX = {"int8": np.float32(127), "e4m3": np.float32(448)}
FITS = {"int8": np.float32(127.5), "e4m3": np.float32(464)}


def e4m3_table():
    """The values of the 256 codes (NaN at 0x7f and 0xff), from the format's definition."""
    out = np.zeros(256, np.float64)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        v = m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        out[c] = np.nan if (c & 0x7F) == 0x7F else (-v if c & 0x80 else v)
    return out


_TABLE = e4m3_table()
_POS = _TABLE[:0x7F]                                   # ascending, codes 0 .. 0x7e
_MID = (_POS[1:] + _POS[:-1]) / 2                      # exact in fp64


def e4m3_encode(y):
    """Codes nearest to y (ties to the even code, saturated), of fp64 values."""
    a = np.abs(np.asarray(y, np.float64))
    lo = np.searchsorted(_MID, a, side="left")         # midpoints below a
    tie = (lo < len(_MID)) & (a == _MID[np.minimum(lo, len(_MID) - 1)])
    code = np.where(tie & (lo % 2 == 1), lo + 1, lo)
    return (code | np.where(np.signbit(y), 0x80, 0)).astype(np.uint8)


def encode(y, kind):
    """fp64 values in units of the scale -> codes (int8, or uint8 holding e4m3)."""
    if kind == "int8":
        return np.clip(np.rint(y), -127, 127).astype(np.int8)
    return e4m3_encode(y)


def values(codes, kind):
    """Codes -> fp64 values in units of the scale."""
    return codes.astype(np.float64) if kind == "int8" else _TABLE[codes]


def grown_scale(s_old, a, kind):
    """(s, k): the scale after doublings that make magnitude a fit, and their number."""
    limit, k = FITS[kind] * np.float32(s_old), 0
    while np.float64(a) > np.float64(limit) * 2.0 ** k:
        k += 1
    return np.float32(np.float64(s_old) * 2.0 ** k), k


class BlockPool:
    """Host model of a block-scaled pool; arrays are the raw regions."""

    def __init__(self, n_layers, n_kv_heads, head_dim, gs, page_size, n_pages, kind):
        assert page_size % gs == 0
        self.n_kv_heads, self.head_dim, self.gs = n_kv_heads, head_dim, gs
        self.page_size, self.n_pages, self.kind = page_size, n_pages, kind
        body = (n_layers, n_pages, n_kv_heads, page_size, head_dim)
        dt = np.int8 if kind == "int8" else np.uint8
        self.k_store, self.v_store = np.zeros(body, dt), np.zeros(body, dt)
        sc = (n_layers, n_pages, n_kv_heads, page_size // gs)
        self.k_scales, self.v_scales = np.zeros(sc, np.float32), np.zeros(sc, np.float32)

    def append(self, layer, k_new, v_new, seq_pos, page_table):
        """k_new, v_new: fp16 [n_seqs][n_new][n_kv_heads][head_dim] behind seq_pos[b] positions.
        Tokens at negative positions, or whose page is not in the table or pool, are left out."""
        gs, ps, kind = self.gs, self.page_size, self.kind
        for new, store, scales in ((k_new, self.k_store, self.k_scales),
                                   (v_new, self.v_store, self.v_scales)):
            new = np.asarray(new, np.float16).astype(np.float32)
            for b in range(new.shape[0]):
                i = max(0, -int(seq_pos[b]))
                while i < new.shape[1]:
                    pos = int(seq_pos[b]) + i
                    n = min(gs - pos % gs, new.shape[1] - i)
                    lp = pos // ps
                    page = int(page_table[b][lp]) if lp < len(page_table[b]) else -1
                    if 0 <= page < self.n_pages:
                        for h in range(self.n_kv_heads):
                            self._block(store[layer, page, h], scales[layer, page, h], pos % ps,
                                        new[b, i:i + n, h])
                    i += n

    def _block(self, rows, scales, slot, x):
        gs, kind = self.gs, self.kind
        blk, r0 = slot // gs, slot % gs
        a = np.max(np.abs(x))
        if r0 and scales[blk] > 0:
            s, k = grown_scale(scales[blk], a, kind)
            if k:
                old = rows[slot - r0:slot]
                old[:] = encode(values(old, kind) * 2.0 ** -k, kind)
        else:
            s = a / QMAX[kind]                                     # fp32 division
        scales[blk] = s
        with np.errstate(divide="ignore", invalid="ignore"):
            y = np.where(s > 0, x / s, np.float32(0))              # fp32 division
        rows[slot:slot + len(x)] = encode(y.astype(np.float64), kind)

    def gather(self, layer, page_table_row, length):
        """Exact fp64 K^, V^ [length][n_kv_heads][head_dim] of positions 0..length-1."""
        pos = np.arange(length)
        pages = np.asarray(page_table_row, np.int64)[pos // self.page_size]
        slots = pos % self.page_size
        out = []
        for store, scales in ((self.k_store, self.k_scales), (self.v_store, self.v_scales)):
            c = values(store[layer, pages, :, slots, :], self.kind)
            s = scales[layer, pages, :, slots // self.gs].astype(np.float64)
            out.append(c * s[..., None])
        return out[0], out[1]
