"""Measured operators around a decoding step: rotation on the way into the cache, attention with
capped, biased or prefix-masked scores over it, and the verification of drafted tokens.

Each in a plain form (elementary torch operations) and through the package's entry points:

* ``rope``: queries and keys of new tokens are rotated by their positions (cosines and sines from a
  table, one position or one for each of three axes); queries come back as fp16, keys and values
  become 8-bit codes in a paged cache: int8 or e4m3 with one fp32 scale for each (block of positions,
  kv head), or int8 rows with fp16 scales (``rows``).  Sequences may bring fewer tokens than others.
* ``scored``: softmax attention of one query, a window of queries, or a whole chunk over a
  block-scaled cache, with scores capped by a tanh, a bias that falls with the distance, a prefix
  that every query sees, and a sliding window.
* ``verify``: how many drafted tokens the target's probabilities accept, and the token behind them,
  from given random numbers.

A case is a dict of plain values; lengths that vary within a batch come from the seed.
"""

import math

import torch

own = False

QMAX = {"int8": 127.0, "e4m3": 448.0}     # largest code
FITS = {"int8": 127.5, "e4m3": 464.0}     # largest |x| / scale that rounds to it


# ---- cases -----------------------------------------------------------------

def listed():
    return [
        # one decoding step of a batch: a token for each of 64 sequences
        dict(name="rope_token", op="rope", kind="int8", seqs=64, n_new=1, ragged=False,
             max_pos=8191, heads=32, heads_kv=8, head_dim=128, page=64, block=64, rot=128,
             style="halves", axes=1),
        # a verify window of five tokens, ragged, on the cache with a scale for each row
        dict(name="rope_rows_window", op="rope", kind="rows", seqs=12, n_new=5, ragged=True,
             max_pos=8191, heads=16, heads_kv=2, head_dim=256, page=64, block=64, rot=64,
             style="pairs", axes=1),
        # a prompt of text and images: three axes, an odd number of tokens behind cached ones
        dict(name="rope_prompt", op="rope", kind="e4m3", seqs=2, n_new=16381, ragged=False,
             max_pos=999, heads=32, heads_kv=8, head_dim=128, page=64, block=32, rot=128,
             style="halves", axes=3),
        # latency: a single user's step at 8K with capped scores
        dict(name="scored_step_8k", op="scored", kind="int8", batch=1, q_len=1, heads=16,
             heads_kv=2, head_dim=256, page=64, block=64, min_len=8192, max_len=8192, empty=0,
             window=0, prefix=0, cap=50.0, slopes=False),
        # throughput: 64 sequences of 1K to 32K with capped scores
        dict(name="scored_batch", op="scored", kind="e4m3", batch=64, q_len=1, heads=32,
             heads_kv=8, head_dim=128, page=64, block=64, min_len=1024, max_len=32768, empty=0,
             window=0, prefix=0, cap=30.0, slopes=False),
        # windows of drafts over long contexts: the last 4096 positions and the first four, biased
        # by distance
        dict(name="scored_window", op="scored", kind="int8", batch=16, q_len=5, heads=32,
             heads_kv=8, head_dim=128, page=32, block=32, min_len=3, max_len=32768, empty=1,
             window=4096, prefix=4, cap=0.0, slopes=True),
        # a chunk of a long prompt with capped scores
        dict(name="scored_chunk", op="chunk", kind="int8", n_new=256, start=32768, heads=16,
             heads_kv=2, head_dim=256, page=64, block=64, window=0, prefix=0, cap=50.0,
             slopes=False),
        # a prompt's start whose first 509 positions see each other, biased by distance
        dict(name="scored_chunk_prefix", op="chunk", kind="e4m3", n_new=1021, start=0, heads=32,
             heads_kv=8, head_dim=128, page=64, block=64, window=0, prefix=509, cap=0.0,
             slopes=True),
        # latency: one user's four drafts
        dict(name="verify_one", op="verify", batch=1, n_draft=4, vocab=32000, drafts=True,
             ragged=False),
        # a batch with a large vocabulary
        dict(name="verify_batch", op="verify", batch=64, n_draft=4, vocab=131072, drafts=True,
             ragged=False),
        # drafts looked up in the text (no probabilities of their own), odd rows, ragged
        dict(name="verify_lookup", op="verify", batch=48, n_draft=7, vocab=50001, drafts=False,
             ragged=True),
    ]


def _log(rng, a, b):
    """An integer in [a, b], spread over its logarithm."""
    return max(a, min(b, int(math.exp(rng.uniform(math.log(a), math.log(b + 1))))))


def draw(rng):
    op = rng.choice(["rope", "rope", "scored", "scored", "chunk", "verify"])
    if op == "verify":
        c = dict(op=op, n_draft=rng.randint(1, 8), vocab=_log(rng, 500, 160000),
                 drafts=rng.random() < 0.7, ragged=rng.random() < 0.5)
        c["batch"] = _log(rng, 1, max(1, min(128, (1 << 25) // (c["vocab"] * (c["n_draft"] + 1)))))
        return c
    c = dict(op=op, kind=rng.choice(["int8", "e4m3"]), heads_kv=rng.choice([1, 2, 3, 4, 8]),
             head_dim=rng.choice([64, 128, 256]), page=rng.choice([16, 32, 64, 128]))
    c["heads"] = c["heads_kv"] * rng.randint(1, 8)
    c["block"] = rng.choice([b for b in (16, 32, 64, 128) if b <= c["page"]])
    row = c["heads_kv"] * c["head_dim"]
    if op == "rope":
        c["kind"] = rng.choice(["int8", "e4m3", "rows"])
        if c["kind"] == "rows":
            c["block"] = rng.choice([b for b in (32, 64, 128, 256) if b <= c["head_dim"]])
        c["rot"] = rng.choice([c["head_dim"], c["head_dim"], c["head_dim"] // 2,
                               16 * rng.randint(1, c["head_dim"] // 16)])
        c["style"] = rng.choice(["halves", "pairs"])
        c["axes"] = rng.choice([1, 1, 3])
        c["ragged"] = rng.random() < 0.4
        c["n_new"] = _log(rng, 1, 8192)
        c["max_pos"] = _log(rng, 1, 8192)
        tokens = (1 << 26) // (c["heads"] * c["head_dim"])
        c["seqs"] = _log(rng, 1, max(1, min(128, tokens // c["n_new"],
                                            (1 << 28) // (row * (c["n_new"] + c["max_pos"])))))
        c["n_new"] = max(1, min(c["n_new"], tokens // c["seqs"]))
        return c
    c["cap"] = rng.choice([0.0, 20.0, 30.0, 50.0])
    c["slopes"] = rng.random() < 0.4 or c["cap"] == 0.0
    c["prefix"] = rng.choice([0, 4, _log(rng, 1, 2000)])
    c["window"] = rng.choice([0, 0, _log(rng, 1, 4096)])
    if op == "chunk":
        c["n_new"] = _log(rng, 1, 1024)
        pairs = (1 << 36) // (c["heads"] * c["head_dim"] * c["n_new"])
        c["start"] = rng.choice([0, _log(rng, 1, max(1, min(32768, pairs)))])
    else:
        c["q_len"] = rng.choice([1, 1, 1, 2, 3, 5, 8])
        c["max_len"] = _log(rng, 1, 131072)
        c["batch"] = _log(rng, 1, max(1, min(128, (1 << 28) // (row * c["max_len"]))))
        c["min_len"] = rng.randint(0, c["max_len"])
        c["empty"] = rng.choice([0, 0, 1])
    return c


# ---- inputs ----------------------------------------------------------------

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _host(seed):
    return torch.Generator().manual_seed(int(seed) * 2654435761 % (1 << 62) + 17)


def _codes(x, kind):
    """fp32 values in units of the scale -> codes."""
    if kind == "e4m3":
        return x.clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
    return x.round().clamp(-127, 127).to(torch.int8)


def _bytes(t):
    return t.view(torch.uint8)


def _quotient(amax, kind):
    """amax / the largest code, correctly rounded (a product with the reciprocal is not)."""
    return amax / torch.full_like(amax, QMAX[kind])


def _cache(c, g, n_pages, used=None):
    """K codes, K scales, V codes, V scales of n_pages pages of normal values; four channels of K are
    outliers.  `used` [n_pages]: rows of a page that hold tokens (the others are zero)."""
    out = []
    for outliers in (True, False):
        x = torch.randn((n_pages, c["heads_kv"], c["page"], c["head_dim"]), generator=g,
                        device="cuda")
        if outliers:
            x[..., :4] *= 20.0
        if used is not None:
            x *= (torch.arange(c["page"], device="cuda")[None, :] < used[:, None])[:, None, :, None]
        x = x.half().float()
        if c["kind"] == "rows":
            b = x.reshape(*x.shape[:3], -1, c["block"])
            s = _quotient(b.abs().amax(dim=-1), "int8").half()
            y = torch.where(s[..., None] > 0, b / s.float()[..., None], torch.zeros_like(b))
            out += [_codes(y, "int8").reshape(x.shape), s]
        else:
            b = x.reshape(*x.shape[:2], -1, c["block"], x.shape[3])
            s = _quotient(b.abs().amax(dim=(3, 4)), c["kind"])
            y = torch.where(s[..., None, None] > 0, b / s[..., None, None], torch.zeros_like(b))
            out += [_codes(y, c["kind"]).reshape(x.shape), s]
    return out


def _table(need, n_pages, width, gen):
    """Page table [rows][width] that gives row r need[r] pages of a seeded permutation, -1 behind."""
    have = torch.arange(width)[None, :] < need[:, None]
    table = torch.full(have.shape, -1, dtype=torch.int32)
    ids = torch.randperm(n_pages, generator=gen).to(torch.int32)
    table[have] = ids[:int(have.sum())]
    return table


def _pages_of(lens, page):
    return (lens + page - 1) // page


def _lengths(lo, hi, n, gen):
    return torch.randint(lo, hi + 1, (n,), generator=gen)


def _slopes(heads):
    return torch.exp2(-8.0 * torch.arange(1, heads + 1, device="cuda") / heads)


def _prepare_rope(c, g, h):
    page, S, n, D = c["page"], c["seqs"], c["n_new"], c["head_dim"]
    pos = _lengths(0, c["max_pos"], S, h)
    lens = _lengths(0, n, S, h) if c["ragged"] else torch.full((S,), n)
    need = _pages_of(pos + lens, page)
    width = -(-(c["max_pos"] + n) // page)
    n_pages = S * width + 1
    table = _table(need, n_pages - 1, width, h)
    used = torch.full((n_pages,), 0)
    held = (pos[:, None] - torch.arange(width)[None, :] * page).clamp(0, page)
    used[table[table >= 0].long()] = held[table >= 0]
    cache = _cache(c, g, n_pages, used.cuda())
    q = torch.randn((S, n, c["heads"], D), generator=g, device="cuda").half()
    k = torch.randn((S, n, c["heads_kv"], D), generator=g, device="cuda")
    k[..., :4] *= 20.0
    v = torch.randn(k.shape, generator=g, device="cuda").half()
    # angles of far positions in 64 bits
    rows = c["max_pos"] + n
    half = c["rot"] // 2
    angle = (torch.arange(rows, device="cuda").double()[:, None]
             * 10000.0 ** (-torch.arange(half, device="cuda").double() / half))
    st = dict(q=q, k_new=k.half(), v_new=v, pos=pos.int().cuda(), table=table.cuda(),
              rope=torch.cat([angle.cos(), angle.sin()], dim=1).float(),
              q_out=torch.zeros_like(q), new_lens=lens.int().cuda() if c["ragged"] else None,
              positions=None, pair_axis=None, axis=None)
    if c["axes"] == 3:      # images of 16 x 16 patches: time stands still, height and width run
        i = torch.arange(n)
        by = torch.stack([i // 256 * 16, i // 256 * 16 + i // 16 % 16, i // 256 * 16 + i % 16])
        st["positions"] = (pos[None, :, None] + by[:, None, :]).int().cuda()
        st["pair_axis"] = (3 * torch.arange(half) // half).to(torch.uint8)       # (kept on the host)
        st["axis"] = st["pair_axis"].long().cuda()
    return st, cache, n_pages


def _prepare_scored(c, g, h):
    page = c["page"]
    if c["op"] == "chunk":
        lens = torch.tensor([c["start"] + c["n_new"]])
        shape = (c["n_new"], c["heads"], c["head_dim"])
        width = int(_pages_of(lens, page)[0])
        prefix = lens.clamp(max=c["prefix"])
    else:
        lens = _lengths(c["min_len"], c["max_len"], c["batch"], h)
        if c["empty"] and c["batch"] > c["empty"]:
            lens[:c["empty"]] = 0
        shape = (c["batch"], c["q_len"], c["heads"], c["head_dim"])
        width = max(1, -(-c["max_len"] // page))
        prefix = torch.full_like(lens, c["prefix"])
    need = _pages_of(lens, page)
    n_pages = 1 + int(need.sum())
    table = _table(need, n_pages - 1, width, h)
    cache = _cache(c, g, n_pages)
    q = torch.randn(shape, generator=g, device="cuda").half()
    st = dict(q=q, out=torch.empty(shape, device="cuda"), lens=lens.int().cuda(),
              table=table.cuda(), slopes=_slopes(c["heads"]) if c["slopes"] else None,
              prefix=prefix.int().cuda())
    return st, cache, n_pages


def _prepare_verify(c, g, h):
    B, n, V = c["batch"], c["n_draft"], c["vocab"]
    logits = 3.0 * torch.randn((B, n + 1, V), generator=g, device="cuda")
    st = dict(target=torch.softmax(logits, dim=2), draft=None,
              u=torch.rand((B, n), generator=g, device="cuda"),
              sample=torch.rand((B,), generator=g, device="cuda"),
              lens=(100 + _lengths(n + 1, 5000, B, h)).int().cuda(),
              n_drafts=_lengths(0, n, B, h).int().cuda() if c["ragged"] else None,
              tokens=torch.empty((B, n + 1), dtype=torch.int32, device="cuda"),
              accepted=torch.empty((B,), dtype=torch.int32, device="cuda"),
              lens_out=torch.empty((B,), dtype=torch.int32, device="cuda"))
    near = logits[:, :n]
    near += torch.randn(near.shape, generator=g, device="cuda")     # the draft model: nearly the same
    if c["drafts"]:
        st["draft"] = torch.softmax(near, dim=2)
        near -= torch.log(-torch.log(torch.rand(near.shape, generator=g, device="cuda")
                                     .clamp(1e-9, 1 - 1e-7)))       # a token drawn from it
    st["x"] = near.argmax(dim=2).int()
    return st


def prepare(case, seed):
    c, g, h = dict(case), _gen(seed), _host(seed)
    if c["op"] == "verify":
        return dict(case=c, **_prepare_verify(c, g, h))
    st, (k, ks, v, vs), n_pages = (_prepare_rope if c["op"] == "rope" else _prepare_scored)(c, g, h)
    if own:       # the pool's handle, and the workspace that a program keeps
        from int8_kv_cache_02_gb300 import binding
        variant = {"int8": "k8v8_block", "e4m3": "f8_block", "rows": "k8v8"}[c["kind"]]
        pool = binding.KVPool(1, c["heads_kv"], c["head_dim"], c["block"], c["page"], n_pages,
                              variant)
        for mine, made in ((pool.k_store, k), (pool.v_store, v), (pool.k_scales, ks),
                           (pool.v_scales, vs)):
            _bytes(mine).copy_(_bytes(made)[None])
        k, ks, v, vs = pool.k_store[0], pool.k_scales[0], pool.v_store[0], pool.v_scales[0]
        st["pool"] = pool
        seen = c["window"] + c["prefix"] if c.get("window") else 1 << 30
        if c["op"] == "scored":
            groups = -(-c["q_len"] * (c["heads"] // c["heads_kv"]) // 8)
            st["splits"] = binding.attn_decode_n_splits(pool, c["batch"] * groups,
                                                        min(c["max_len"], seen))
            st["workspace"] = pool.decode_workspace(c["batch"] * c["q_len"], c["heads"],
                                                    st["splits"])
        elif c["op"] == "chunk":
            st["splits"] = binding.attn_prefill_n_splits(pool, c["n_new"], c["heads"],
                                                         min(c["start"], seen))
            n = binding.attn_prefill_workspace_bytes(c["n_new"], c["heads"], c["heads_kv"],
                                                     c["head_dim"], st["splits"])
            st["workspace"] = torch.empty(max(n, 16), dtype=torch.uint8, device="cuda")
    return dict(st, case=c, k=k, ks=ks, v=v, vs=vs)


# ---- plain forms -----------------------------------------------------------

def _pow2(k):
    """2 ** k as fp32, exactly, for whole numbers k."""
    return ((k.clamp(-126, 127) + 127).int() << 23).view(torch.float32)


def _rotated(x, st):
    """[S][n][heads][D] fp16 -> fp32, pairs of the first `rot` values turned."""
    c = st["case"]
    x, half = x.float(), c["rot"] // 2
    S, n = x.shape[:2]
    if st["positions"] is None:
        at = st["pos"].long()[:, None] + torch.arange(n, device=x.device)
        cs = st["rope"][at]                                                # [S][n][rot]
        cos, sin = cs[..., :half], cs[..., half:]
    else:
        pair = torch.arange(half, device=x.device)
        at = st["positions"].long()[st["axis"]].permute(1, 2, 0)                 # [S][n][half]
        cos, sin = st["rope"][at, pair], st["rope"][at, half + pair]
    cos, sin = cos[:, :, None], sin[:, :, None]
    if c["style"] == "halves":
        a, b = x[..., :half], x[..., half:2 * half]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], dim=3)
    else:
        a, b = x[..., 0:2 * half:2], x[..., 1:2 * half:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], dim=4).flatten(3)
    return torch.cat([turned, x[..., 2 * half:]], dim=3)


def _append_blocks(store, scales, x, lens, st):
    """x [S][n][H][D] fp32, the first lens[s] tokens of each behind pos[s] cached ones."""
    c = st["case"]
    T, page, kind = c["block"], c["page"], c["kind"]
    S, n, H, D = x.shape
    pos, table = st["pos"].long(), st["table"].long()
    row_of, scale_of = _bytes(store).reshape(-1, D), scales.reshape(-1)
    per_page, spare = page // T, store.shape[0] - 1     # the last page is no sequence's
    nb = (n + T - 2) // T + 1                           # blocks that n tokens may touch
    off = pos % T
    i = torch.arange(n, device=x.device)
    new = i < lens[:, None]                             # [S][n]
    at = off[:, None] + i
    amax = torch.zeros((S, nb, H), device=x.device)
    top = x.abs().amax(dim=3).masked_fill(~new[..., None], 0.0)
    amax.scatter_reduce_(1, (at // T)[..., None].expand(S, n, H), top, "amax")
    first = (pos // T)[:, None] + torch.arange(nb, device=x.device)
    touched = first * T < (pos + lens)[:, None]
    pg = table.gather(1, (first // per_page).clamp(max=table.shape[1] - 1))
    pg = torch.where(touched, pg, spare)
    slot = ((pg[..., None] * H + torch.arange(H, device=x.device)) * per_page
            + (first % per_page)[..., None])            # [S][nb][H]
    old = scale_of[slot]
    held = (off > 0)[:, None, None] & (torch.arange(nb, device=x.device) == 0)[None, :, None]
    held = held & (old > 0)
    ma, ea = torch.frexp(amax)
    ml, el = torch.frexp(old * FITS[kind])
    up = torch.where(held & (amax > 0), (ea - el + (ma > ml)).clamp(min=0), torch.zeros_like(ea))
    s = torch.where(held, old * _pow2(up), _quotient(amax, kind))
    s = torch.where(touched[..., None], s, old)
    scale_of.index_put_((slot,), s)
    # the rows that the first block held already
    r = ((pg[:, 0, None, None] * H + torch.arange(H, device=x.device)[None, :, None]) * page
         + ((first[:, 0] % per_page) * T)[:, None, None] + torch.arange(T, device=x.device))
    was = row_of[r].view(store.dtype)
    less = _codes(was.float() * _pow2(-up[:, 0, :, None, None]), kind)
    keep = (torch.arange(T, device=x.device) >= off[:, None])[:, None, :, None]
    row_of.index_put_((r,), torch.where(keep, _bytes(was), _bytes(less)))
    # the new rows (a token that is none writes the spare page's first rows as they are)
    sx = s.gather(1, (at // T)[..., None].expand(S, n, H))[..., None]
    y = _codes(torch.where(sx > 0, x / sx, torch.zeros_like(x)), kind)
    _put_rows(row_of, _bytes(y), new, pos, table, spare, page)


def _put_rows(row_of, y, new, pos, table, spare, page):
    S, n, H = y.shape[:3]
    tok = pos[:, None] + torch.arange(n, device=y.device)
    pt = torch.where(new, table.gather(1, (tok // page).clamp(max=table.shape[1] - 1)), spare)
    slot = torch.where(new, tok % page, 0)
    r = (pt[..., None] * H + torch.arange(H, device=y.device)) * page + slot[..., None]
    row_of.index_put_((r,), torch.where(new[..., None, None], y, row_of[r]))


def _append_rows(store, scales, x, lens, st):
    """The same into the cache with fp16 scales of `block` values of a row."""
    c = st["case"]
    b = x.reshape(*x.shape[:3], -1, c["block"])
    s = _quotient(b.abs().amax(dim=-1), "int8").half()
    y = torch.where(s[..., None] > 0, b / s.float()[..., None], torch.zeros_like(b))
    y = _codes(y, "int8").reshape(x.shape)
    new = torch.arange(x.shape[1], device=x.device) < lens[:, None]
    args = (new, st["pos"].long(), st["table"].long(), store.shape[0] - 1, c["page"])
    _put_rows(_bytes(store).reshape(-1, x.shape[3]), _bytes(y), *args)
    _put_rows(scales.reshape(-1, s.shape[3]), s, *args)


def _rope(st):
    c = st["case"]
    n = c["n_new"]
    lens = st["new_lens"]
    lens = torch.full_like(st["pos"], n).long() if lens is None else lens.long()
    new = (torch.arange(n, device=lens.device) < lens[:, None])[..., None, None]
    st["q_out"].copy_(torch.where(new, _rotated(st["q"], st).half(), st["q_out"]))
    append = _append_rows if c["kind"] == "rows" else _append_blocks
    append(st["k"], st["ks"], _rotated(st["k_new"], st), lens, st)
    append(st["v"], st["vs"], st["v_new"].float(), lens, st)


def _scored(st):
    c = st["case"]
    chunk = c["op"] == "chunk"
    q, table, lens = st["q"][None] if chunk else st["q"], st["table"].long().clamp(min=0), \
        st["lens"].long()
    B, Q, Hq, D = q.shape
    H, page, T = c["heads_kv"], c["page"], c["block"]
    n = table.shape[1] * page
    pos = torch.arange(n, device=q.device)

    def gathered(store, scales):
        x = _bytes(store)[table].view(store.dtype).float()               # [B][pages][H][page][D]
        x = x.reshape(B, -1, H, page // T, T, D) * scales[table][..., None, None]
        return x.reshape(B, -1, H, page, D).transpose(1, 2).reshape(B, H, n, D)

    last = lens[:, None] - Q + torch.arange(Q, device=q.device)          # [B][Q]
    seen = pos <= last[..., None]
    if c["window"]:
        seen &= pos > last[..., None] - c["window"]
    seen |= pos < st["prefix"].long()[:, None, None]
    seen &= (pos < lens[:, None])[:, None, :] & (last >= 0)[..., None]
    x = q.float().reshape(B, Q, H, Hq // H, D).transpose(1, 2).reshape(B, H, -1, D)
    s = ((x / math.sqrt(D)) @ gathered(st["k"], st["ks"]).transpose(2, 3))
    s = s.reshape(B, H, Q, Hq // H, n)
    if c["cap"]:
        s = torch.tanh(s / c["cap"]) * c["cap"]
    if c["slopes"]:
        s += (st["slopes"].reshape(1, H, 1, Hq // H, 1)
              * (pos - last[..., None]).float()[:, None, :, None, :])
    s = s.masked_fill(~seen[:, None, :, None, :], -math.inf)
    m = s.amax(dim=-1, keepdim=True)
    p = torch.exp(s - torch.where(m > -math.inf, m, torch.zeros_like(m)))
    l = p.sum(dim=-1, keepdim=True)
    v = gathered(st["v"], st["vs"])
    v = v.masked_fill((pos >= lens[:, None])[:, None, :, None], 0.0)
    o = (p / torch.where(l > 0, l, torch.ones_like(l))).reshape(B, H, -1, n) @ v
    o = o.reshape(B, H, Q, Hq // H, D).transpose(1, 2).reshape(B, Q, Hq, D)
    return o[0] if chunk else o


def _verify(st):
    """In 64 bits: a comparison of two products, and long sums that a border is looked up in."""
    p, q, x = st["target"], st["draft"], st["x"].long()
    B, n = x.shape
    i = torch.arange(n, device=x.device)
    count = torch.full((B,), n, device=x.device) if st["n_drafts"] is None else \
        st["n_drafts"].long()
    px = p[:, :n].gather(2, x[..., None])[..., 0].double()
    qx = torch.ones_like(px) if q is None else q.gather(2, x[..., None])[..., 0].double()
    take = (st["u"].double() * qx < px) & (i < count[:, None])
    accepted = take.long().cumprod(dim=1).sum(dim=1)
    rows = torch.arange(B, device=x.device)
    refused = accepted < count
    at = accepted.clamp(max=n - 1)
    pw = p[rows, accepted].double()
    if q is None:
        qw = torch.zeros_like(pw).scatter_(1, x[rows, at][:, None], 1.0)
    else:
        qw = q[rows, at].double()
    w = torch.where(refused[:, None], (pw - qw).clamp(min=0.0), pw)
    w = torch.where((w.sum(dim=1) > 0)[:, None], w, pw)
    c = w.cumsum(dim=1)
    above = c > st["sample"].double()[:, None] * c[:, -1:]
    token = torch.where(above.any(dim=1), above.int().argmax(dim=1), -1)
    j = torch.arange(n + 1, device=x.device)
    out = torch.cat([x, torch.full((B, 1), -1, device=x.device)], dim=1)
    out = torch.where(j < accepted[:, None], out, torch.full_like(out, -1))
    out.scatter_(1, accepted[:, None], token[:, None])
    st["tokens"].copy_(out)
    st["accepted"].copy_(accepted)
    st["lens_out"].copy_(st["lens"] - (count - accepted).int())


# ---- one pass --------------------------------------------------------------

def run(st):
    c = st["case"]
    if own:
        from int8_kv_cache_02_gb300 import binding
    if c["op"] == "rope":
        if own:
            binding.kv_rope_append(st["pool"], 0, st["k_new"], st["v_new"], st["pos"], st["table"],
                                   st["rope"], q=st["q"], q_out=st["q_out"],
                                   positions=st["positions"], pair_axis=st["pair_axis"],
                                   rope_dim=c["rot"], style=c["style"], new_lens=st["new_lens"])
        else:
            _rope(st)
        return dict(q=st["q_out"], k=st["k"], ks=st["ks"], v=st["v"], vs=st["vs"])
    if c["op"] == "verify":
        if own:
            binding.kv_verify_drafts(st["target"], st["x"], st["u"], st["sample"], st["tokens"],
                                     st["accepted"], draft_probs=st["draft"],
                                     n_drafts=st["n_drafts"], seq_lens=st["lens"],
                                     seq_lens_out=st["lens_out"])
        else:
            _verify(st)
        return dict(tokens=st["tokens"], accepted=st["accepted"], lens=st["lens_out"])
    if not own:
        return _scored(st)
    if c["op"] == "chunk":
        binding.attn_prefill_chunk_scored_int8(
            st["pool"], 0, st["q"], c["start"], st["table"], st["out"], st["workspace"],
            window=c["window"], softcap=c["cap"], slopes=st["slopes"], prefix_len=c["prefix"],
            n_splits=st["splits"])
    else:
        binding.attn_decode_scored_int8(
            st["pool"], 0, st["q"], st["lens"], st["table"], st["out"], st["workspace"],
            window=c["window"], softcap=c["cap"], slopes=st["slopes"],
            prefix_lens=st["prefix"] if c["prefix"] else None, n_splits=st["splits"])
    return st["out"]


# ---- what a pass cannot do without -----------------------------------------

def _seen_by(c, length, rows):
    """Visible positions, summed over `rows` queries that end a context of `length`."""
    total = 0.0
    for i in (0.5,) if rows > 64 else range(rows):     # (the middle query stands for many)
        last = length - rows + (rows * i if rows > 64 else i)
        own_part = min(last + 1, c["window"]) if c["window"] else last + 1
        total += max(0.0, min(length, own_part + min(max(c["prefix"] - (last + 1 - own_part), 0)
                                                     if c["prefix"] > last else c["prefix"],
                                                     length - own_part)))
    return total * rows if rows > 64 else total


def work(case):
    c = case
    if c["op"] == "verify":
        B, n, V = c["batch"], c["n_draft"], c["vocab"]
        rows = 2 if c["drafts"] else 1
        return {"bytes": B * (4 * rows * V + 4 * (5 * n + 6)), "flops": B * rows * V}
    H, Hkv, D = c["heads"], c["heads_kv"], c["head_dim"]
    row = 2 * Hkv * D                                      # K and V codes of one token
    if c["op"] == "rope":
        n = c["seqs"] * c["n_new"] * (0.5 if c["ragged"] else 1.0)
        scales = (4 * Hkv * D / c["block"] if c["kind"] == "rows" else 8 * Hkv / c["block"])
        return {"bytes": n * (3 * row + 4 * H * D + 4 * c["rot"] + scales) + 8 * c["seqs"],
                "flops": 3 * n * (H + Hkv) * c["rot"] + 2 * n * row}
    if c["op"] == "chunk":
        length, batch, rows = c["start"] + c["n_new"], 1, c["n_new"]
        tokens = min(length, c["window"] + rows + c["prefix"]) if c["window"] else length
    else:
        length, rows = (c["min_len"] + c["max_len"]) / 2, c["q_len"]     # the seed decides: their mean
        batch = c["batch"] - (c["empty"] if c["batch"] > c["empty"] else 0)
        tokens = min(length, c["window"] + rows + c["prefix"]) if c["window"] else length
    io = batch * rows * H * D * (2 + 4)
    return {"bytes": batch * tokens * (row + 8 * Hkv / c["block"] + 4 / c["page"]) + io + 4 * batch,
            "flops": 4 * batch * _seen_by(c, length, rows) * H * D + 1}


# ---- the definitions in 64 bits --------------------------------------------

def _exact_turned(x, st):
    """One token after the other's positions, pair by pair, in 64 bits."""
    c = st["case"]
    x, half = x.double().clone(), c["rot"] // 2
    n, rope = x.shape[1], st["rope"].double()
    for i in range(half):
        axis = int(st["pair_axis"][i]) if st["pair_axis"] is not None else 0
        at = (st["positions"][axis].long() if st["positions"] is not None else
              st["pos"].long()[:, None] + torch.arange(n, device=x.device)[None, :])
        co, si = rope[at, i][..., None], rope[at, half + i][..., None]
        ia, ib = (i, i + half) if c["style"] == "halves" else (2 * i, 2 * i + 1)
        a, b = x[..., ia].clone(), x[..., ib].clone()
        x[..., ia] = a * co - b * si
        x[..., ib] = a * si + b * co
    return x


def _exact_blocks(codes, scales, x, lens, st):
    """One store [pages][heads][page][D] in 64 bits (values in units of the scale) and its scales,
    block by block."""
    c = st["case"]
    T, page, kind = c["block"], c["page"], c["kind"]
    pos, table = st["pos"].tolist(), st["table"].tolist()

    def rounded(y):
        if kind == "int8":
            return torch.clamp(torch.round(y), -127, 127)
        return torch.clamp(y, -448, 448).float().to(torch.float8_e4m3fn).double()

    for b in range(x.shape[0]):
        i = 0
        while i < lens[b]:
            p = pos[b] + i
            n = min(T - p % T, lens[b] - i)
            new = x[b, i:i + n].transpose(0, 1)                             # [heads][n][D]
            top = new.abs().amax(dim=(1, 2))
            pg, r0, blk, at = table[b][p // page], p % T, (p % page) // T, p % page
            s = top / QMAX[kind]
            if r0:
                was = scales[pg, :, blk]
                k = torch.ceil(torch.log2(top / (was * FITS[kind]))).clamp(min=0)
                k = torch.where((was > 0) & (top > 0), k, torch.zeros_like(k))
                s = torch.where(was > 0, was * torch.exp2(k), s)
                lo = at - r0
                codes[pg, :, lo:at] = rounded(codes[pg, :, lo:at] * torch.exp2(-k)[:, None, None])
            scales[pg, :, blk] = s
            codes[pg, :, at:at + n] = rounded(torch.where(s[:, None, None] > 0,
                                                          new / s[:, None, None], new))
            i += n


def _exact_rope(st):
    c = st["case"]
    S, n, page = c["seqs"], c["n_new"], c["page"]
    lens = [n] * S if st["new_lens"] is None else st["new_lens"].tolist()
    q = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
    turned = _exact_turned(st["q"], st)
    for b in range(S):
        q[b, :lens[b]] = turned[b, :lens[b]]
    res = dict(q=q, k=None, v=None)
    for name, new in (("k", _exact_turned(st["k_new"], st)), ("v", st["v_new"].double())):
        codes, scales = st[name].float().double(), st[name + "s"].double()
        if c["kind"] == "rows":
            table, pos = st["table"].tolist(), st["pos"].tolist()
            for b in range(S):
                for i in range(lens[b]):
                    p = pos[b] + i
                    top = new[b, i].reshape(c["heads_kv"], -1, c["block"]).abs().amax(dim=2)
                    scales[table[b][p // page], :, p % page] = top / 127.0
        else:
            _exact_blocks(codes, scales, new, lens, st)
            if c["kind"] == "e4m3":
                res[name] = codes
        res[name + "s"] = scales
    return res


def _exact_scored(st):
    c = st["case"]
    T, page, G = c["block"], c["page"], c["heads"] // c["heads_kv"]
    chunk = c["op"] == "chunk"
    q = (st["q"][None] if chunk else st["q"]).double()
    Q = q.shape[1]
    out = torch.zeros_like(q)
    for b, n in enumerate(st["lens"].tolist()):
        if not n:
            continue
        ids = st["table"][b, :-(-n // page)].long()
        rows = []
        for codes, scales in ((st["k"], st["ks"]), (st["v"], st["vs"])):
            x = _bytes(codes)[ids].view(codes.dtype).float().double()
            x = x * scales[ids].double().repeat_interleave(T, dim=2)[..., None]
            rows.append(x.permute(1, 0, 2, 3).reshape(c["heads_kv"], -1, c["head_dim"])[:, :n])
        j = torch.arange(n, device="cuda")
        for i0 in range(0, Q, 64):      # queries together, as far as memory goes
            here = torch.arange(i0, min(Q, i0 + 64), device="cuda")
            last = (n - Q + here)[:, None]
            hidden = j > last
            if c["window"]:
                hidden |= last - j >= c["window"]
            hidden &= j >= c["prefix"]
            for h in range(c["heads"]):
                s = q[b, here, h] @ rows[0][h // G].T / math.sqrt(c["head_dim"])
                if c["cap"]:
                    s = c["cap"] * torch.tanh(s / c["cap"])
                if c["slopes"]:
                    s = s - float(st["slopes"][h]) * (last - j)
                o = torch.softmax(s.masked_fill(hidden, -math.inf), dim=1) @ rows[1][h // G]
                out[b, here, h] = torch.where(last < 0, torch.zeros_like(o), o)
    return out[0] if chunk else out


def exact(case, seed):
    c = dict(case)
    if c["op"] == "verify":
        return None                       # whole numbers only
    st = prepare(c, seed)
    if c["op"] != "rope":
        return _exact_scored(st)
    blocks = c["seqs"] * (c["n_new"] if c["kind"] == "rows" else 2 + c["n_new"] // c["block"])
    return _exact_rope(st) if blocks <= 20000 else None
