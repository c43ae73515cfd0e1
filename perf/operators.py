"""Measured operators: the block-scaled 8-bit cache, attention over it, and its pages.

Three operators that belong together, each in a plain form (elementary torch
operations) and through the package's entry points:

* ``append``: fp16 K and V rows of new tokens become 8-bit codes (int8 or e4m3)
  with one fp32 scale for each (block of positions, kv head), written through a
  page table.  A block that already holds tokens keeps its scale unless a new
  value does not fit; then the scale doubles until it does and the block's
  older codes are halved as often.
* ``decode``: softmax attention of one query, or of a window of queries that is
  causal within itself, over that cache, with an optional sliding window and an
  optional one-token append in front.
* ``pages``: copying pages, forking sequences, giving every sequence the pages
  its length needs (and taking back the others), and compacting the pool.

A case is a dict of plain values; lengths that vary within a batch come from
the seed.  ``min_len`` and ``max_len`` bound them; ``empty`` of the sequences
hold nothing.
"""

import math

import torch

own = False

QMAX = {"int8": 127.0, "e4m3": 448.0}     # largest code
FITS = {"int8": 127.5, "e4m3": 464.0}     # largest |x| / scale that rounds to it
LOG2E = 1.4426950408889634


# ---- cases -----------------------------------------------------------------

def listed():
    return [
        # one decoding step of a batch: a token for each of 64 sequences
        dict(name="append_token", op="append", kind="int8", seqs=64, n_new=1, max_pos=8191,
             heads_kv=8, head_dim=128, page=64, block=64),
        # a prompt's remaining tokens behind an odd number of cached ones
        dict(name="append_prompt", op="append", kind="e4m3", seqs=2, n_new=16381, max_pos=999,
             heads_kv=8, head_dim=128, page=64, block=32),
        # latency: a single user's step at 8K, the new token's append included
        dict(name="decode_step_8k", op="decode", kind="int8", batch=1, heads=16, heads_kv=2,
             head_dim=256, page=64, block=64, min_len=8192, max_len=8192, empty=0, window=0,
             q_len=1, append=True),
        # a single user's long context
        dict(name="decode_128k", op="decode", kind="int8", batch=1, heads=16, heads_kv=2,
             head_dim=256, page=64, block=64, min_len=131072, max_len=131072, empty=0, window=0,
             q_len=1, append=False),
        # throughput: 64 sequences of 1K to 32K
        dict(name="decode_batch", op="decode", kind="e4m3", batch=64, heads=32, heads_kv=8,
             head_dim=128, page=64, block=64, min_len=1024, max_len=32768, empty=0, window=0,
             q_len=1, append=False),
        # speculative decoding: four queries to verify for each of 12 ragged sequences
        dict(name="decode_verify", op="decode", kind="e4m3", batch=12, heads=32, heads_kv=8,
             head_dim=128, page=32, block=32, min_len=3, max_len=8191, empty=1, window=0,
             q_len=4, append=False),
        # a prefix cache that duplicates pages
        dict(name="pages_copy", op="copy", kind="int8", layers=2, heads_kv=8, head_dim=128,
             page=64, block=64, n_pages=2048, copies=512),
        # sampling: one prompt continued twice
        dict(name="pages_fork_one", op="fork", kind="int8", layers=4, heads_kv=2, head_dim=256,
             page=64, block=64, n_pages=1024, parents=1, per_parent=1, rows=8, max_len=8191),
        # beam search: 16 prompts with four beams each
        dict(name="pages_fork_beams", op="fork", kind="e4m3", layers=2, heads_kv=8, head_dim=128,
             page=64, block=64, n_pages=8192, parents=16, per_parent=4, rows=96, max_len=6001),
        # continuous batching: sequences end, start and grow between two steps
        dict(name="pages_resize", op="resize", kind="int8", layers=1, heads_kv=1, head_dim=64,
             page=16, block=16, n_pages=65536, rows=256, max_len=8191),
        # a pool after long use, gathered at its low end before it is shrunk
        dict(name="pages_compact", op="compact", kind="int8", layers=2, heads_kv=8, head_dim=128,
             page=64, block=64, n_pages=6144, rows=64, max_len=6001),
        # a small pool of one layer
        dict(name="pages_compact_small", op="compact", kind="e4m3", layers=1, heads_kv=2,
             head_dim=128, page=32, block=16, n_pages=512, rows=7, max_len=1000),
    ]


def _log(rng, a, b):
    """An integer in [a, b], spread over its logarithm."""
    return max(a, min(b, int(math.exp(rng.uniform(math.log(a), math.log(b + 1))))))


def draw(rng):
    c = dict(kind=rng.choice(["int8", "e4m3"]), heads_kv=rng.choice([1, 2, 3, 4, 8]),
             head_dim=rng.choice([64, 128, 256]), page=rng.choice([16, 32, 64, 128]))
    c["block"] = rng.choice([b for b in (16, 32, 64, 128) if b <= c["page"]])
    row = c["heads_kv"] * c["head_dim"]
    op = rng.choice(["append", "decode", "decode", "copy", "fork", "resize", "compact"])
    c["op"] = op
    if op == "append":
        c["n_new"] = _log(rng, 1, 8192)
        c["max_pos"] = _log(rng, 1, 8192)
        c["seqs"] = _log(rng, 1, max(1, min(128, (1 << 17) // c["n_new"],
                                            (1 << 28) // (row * (c["n_new"] + c["max_pos"])),
                                            (1 << 25) // (row * c["n_new"]))))
    elif op == "decode":
        c["max_len"] = _log(rng, 1, 131072)
        c["batch"] = _log(rng, 1, max(1, min(128, (1 << 28) // (row * c["max_len"]))))
        c["min_len"] = rng.randint(0, c["max_len"])
        c["heads"] = c["heads_kv"] * rng.randint(1, 8)
        c["empty"] = rng.choice([0, 0, 1])
        c["q_len"] = rng.choice([1, 1, 1, 2, 3, 5, 8])
        c["window"] = _log(rng, 1, 4096) if c["q_len"] == 1 and rng.random() < 0.3 else 0
        c["append"] = c["q_len"] == 1 and c["min_len"] > 0 and rng.random() < 0.3
    else:
        c["layers"] = rng.randint(1, 4)
        c["n_pages"] = _log(rng, 64, max(65, min(65536, (1 << 28) // (row * c["page"] *
                                                                      c["layers"]))))
        if op == "copy":
            c["copies"] = _log(rng, 1, c["n_pages"] // 2)
        else:
            c["rows"] = _log(rng, 4, max(4, min(128, c["n_pages"] // 4)))
            c["max_len"] = _log(rng, 1, max(1, c["n_pages"] * c["page"] // (2 * c["rows"])))
        if op == "fork":
            c["parents"] = rng.randint(1, max(1, c["rows"] // 4))
            c["per_parent"] = rng.randint(1, 3)
    return c


# ---- inputs ----------------------------------------------------------------

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _host(seed):
    return torch.Generator().manual_seed(int(seed) * 2654435761 % (1 << 62) + 17)


def _codes(x, kind):
    """fp32 values in units of the scale -> codes."""
    if kind == "int8":
        return x.round().clamp(-127, 127).to(torch.int8)
    return x.clamp(-448.0, 448.0).to(torch.float8_e4m3fn)


def _values(c):
    """Codes -> the fp32 values they stand for, in units of the scale."""
    return c.to(torch.float32)


def _bytes(t):
    return t.view(torch.uint8)


def _quotient(amax, kind):
    """amax / the largest code, correctly rounded (a product with the reciprocal is not)."""
    return amax / torch.full_like(amax, QMAX[kind])


def _quantised(x, c):
    """[pages][heads][page][head_dim] values -> codes and scales of the cache's blocks."""
    n, h, p, d = x.shape
    b = x.reshape(n, h, p // c["block"], c["block"], d)
    s = _quotient(b.abs().amax(dim=(3, 4)), c["kind"])
    y = torch.where(s[..., None, None] > 0, b / s[..., None, None], torch.zeros_like(b))
    return _codes(y, c["kind"]).reshape(n, h, p, d), s


def _cache(c, g, n_pages, layers=1, used=None):
    """Stores of `layers` x n_pages pages of normal values; four channels of K are outliers.
    `used` [n_pages]: rows of a page that hold tokens (the others are zero)."""
    out = []
    for outliers in (True, False):
        codes, scales = [], []
        for _ in range(layers):
            x = torch.randn((n_pages, c["heads_kv"], c["page"], c["head_dim"]), generator=g,
                            device="cuda")
            if outliers:
                x[..., :4] *= 20.0
            if used is not None:
                x *= (torch.arange(c["page"], device="cuda")[None, :] < used[:, None])[:, None, :,
                                                                                      None]
            q, s = _quantised(x.half().float(), c)
            codes.append(q)
            scales.append(s)
        out += [torch.stack([_bytes(q) for q in codes]).view(codes[0].dtype), torch.stack(scales)]
    return out


def _pow2(k):
    """2 ** k as fp32, exactly, for whole numbers k."""
    return ((k.clamp(-126, 127) + 127).int() << 23).view(torch.float32)


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


def prepare(case, seed):
    c, g, h = dict(case), _gen(seed), _host(seed)
    st = {"case": c}
    op, page = c["op"], c["page"]
    if op == "append":
        pos = _lengths(0, c["max_pos"], c["seqs"], h)
        need = _pages_of(pos + c["n_new"], page)
        width = -(-(c["max_pos"] + c["n_new"]) // page)
        n_pages = c["seqs"] * width + 1
        table = _table(need, n_pages - 1, width, h)
        used = torch.full((n_pages,), 0)
        first = torch.arange(width)[None, :] * page
        held = (pos[:, None] - first).clamp(0, page)
        used[table[table >= 0].long()] = held[table >= 0]
        k, ks, v, vs = _cache(c, g, n_pages, 1, used.cuda())
        shape = (c["seqs"], c["n_new"], c["heads_kv"], c["head_dim"])
        kn = torch.randn(shape, generator=g, device="cuda")
        kn[..., :4] *= 20.0
        vn = torch.randn(shape, generator=g, device="cuda")
        st |= dict(k_new=kn.half(), v_new=vn.half(), pos=pos.int().cuda(), table=table.cuda())
        layers = 1
    elif op == "decode":
        lens = _lengths(c["min_len"], c["max_len"], c["batch"], h)
        if c["empty"] and c["batch"] > c["empty"]:
            lens[:c["empty"]] = 0
        if c["append"]:
            lens = lens.clamp(min=1)
        need = _pages_of(lens, page)
        width = max(1, -(-c["max_len"] // page))
        n_pages = 1 + (c["batch"] * width if c["append"] else int(need.sum()))
        table = _table(need, n_pages - 1, width, h)
        k, ks, v, vs = _cache(c, g, n_pages)
        q = torch.randn((c["batch"], c["q_len"], c["heads"], c["head_dim"]), generator=g,
                        device="cuda").half()
        st |= dict(q=q if c["q_len"] > 1 else q[:, 0].contiguous(), lens=lens.int().cuda(),
                   table=table.cuda(),
                   out=torch.empty(q.shape if c["q_len"] > 1 else q[:, 0].shape, device="cuda"))
        if c["append"]:
            kn = torch.randn((c["batch"], c["heads_kv"], c["head_dim"]), generator=g, device="cuda")
            kn[..., :4] *= 20.0
            st |= dict(k_new=kn.half(), v_new=torch.randn(kn.shape, generator=g,
                                                          device="cuda").half())
        layers = 1
    else:
        n_pages, layers = c["n_pages"], c["layers"]
        k, ks, v, vs = _cache(c, g, n_pages, layers)
        if op == "copy":
            ids = torch.randperm(n_pages, generator=h).int()
            st |= dict(src=ids[:c["copies"]].cuda(),
                       dst=ids[c["copies"]:2 * c["copies"]].contiguous().cuda())
        else:
            rows = c["rows"]
            if op == "fork":
                n = c["parents"] * c["per_parent"]
                rows = max(rows, c["parents"] + n)
            cap = max(1, n_pages * page // rows - page)       # the rows fit the pool
            lens = _lengths(1, max(1, min(c["max_len"], cap // (2 if op == "resize" else 1))),
                            rows, h)
            new = lens
            if op == "resize":       # a quarter ends, a quarter starts, the others grow by one
                part = torch.randperm(rows, generator=h) % 4
                new = torch.where(part == 0, torch.zeros_like(lens), lens + 1)
                lens = torch.where(part == 1, torch.zeros_like(lens), lens)
            need = _pages_of(lens, page)
            width = max(1, -(-(c["max_len"] + 1) // page))
            table = _table(need, n_pages, width, h)
            refs = torch.zeros(n_pages, dtype=torch.int32)
            refs[table[table >= 0].long()] = 1
            if op in ("compact", "resize") and rows >= 4:     # the last row shares the first's
                refs[table[-1][table[-1] >= 0].long()] = 0    # full pages
                table[-1] = -1
                full = int(lens[0]) // page
                table[-1, :full] = table[0, :full]
                refs[table[0, :full].long()] += 1
                lens[-1] = full * page
                if op == "resize":
                    new[-1] = full * page
                    lens[-1] = full * page
            st |= dict(table=table.cuda(), refs=refs.cuda(), lens=lens.int().cuda())
            if op == "resize":
                st["lens"] = new.int().cuda()
            if op == "fork":
                ids = torch.randperm(rows, generator=h).int()
                st |= dict(parents=ids[:c["parents"]].repeat_interleave(c["per_parent"]).cuda(),
                           children=ids[c["parents"]:c["parents"] + n].contiguous().cuda())
            if op == "compact":
                st |= dict(table_out=torch.empty_like(st["table"]),
                           refs_out=torch.empty_like(st["refs"]),
                           n_used=torch.empty(1, dtype=torch.int32, device="cuda"))
    if own:       # the pool's handle, and the workspaces that a program keeps
        from int8_kv_cache_02_gb300 import binding
        pool = binding.KVPool(layers, c["heads_kv"], c["head_dim"], c["block"], page, n_pages,
                              "k8v8_block" if c["kind"] == "int8" else "f8_block")
        for mine, made in ((pool.k_store, k), (pool.v_store, v), (pool.k_scales, ks),
                           (pool.v_scales, vs)):
            _bytes(mine).copy_(_bytes(made))
        k, ks, v, vs = pool.k_store, pool.k_scales, pool.v_store, pool.v_scales
        st["pool"] = pool
        if op == "decode":
            groups = -(-c["q_len"] * (c["heads"] // c["heads_kv"]) // 8)
            st["splits"] = binding.attn_decode_n_splits(pool, c["batch"] * groups, c["max_len"])
            st["workspace"] = pool.decode_workspace(c["batch"] * c["q_len"], c["heads"],
                                                    st["splits"])
        elif op in ("fork", "resize", "compact"):
            st["workspace"] = pool.pages_workspace(st["table"].shape[0])
    st |= dict(k=k, ks=ks, v=v, vs=vs)
    return st


# ---- plain forms -----------------------------------------------------------

def _append_one(store, scales, x, pos, table, c):
    """x [seqs][n][heads][head_dim] behind pos[s] cached tokens, into layer 0 of a store."""
    T, page, kind = c["block"], c["page"], c["kind"]
    S, n, H, D = x.shape
    pos = pos.long()
    row_of = _bytes(store[0]).reshape(-1, D)
    scale_of = scales[0].reshape(-1)
    per_page = page // T
    nb = (n + T - 2) // T + 1                           # blocks that n tokens may touch
    off = pos % T
    x = x.float()
    at = off[:, None] + torch.arange(n, device=x.device)[None, :]
    amax = torch.zeros((S, nb, H), device=x.device)
    amax.scatter_reduce_(1, (at // T)[..., None].expand(S, n, H), x.abs().amax(dim=3), "amax")
    first = (pos // T)[:, None] + torch.arange(nb, device=x.device)[None, :]
    touched = first * T < (pos + n)[:, None]
    pg = table.long().gather(1, (first // per_page).clamp(max=table.shape[1] - 1))
    pg = torch.where(touched, pg, store.shape[1] - 1)   # the last page is no sequence's
    slot = ((pg[..., None] * H + torch.arange(H, device=x.device)) * per_page
            + (first % per_page)[..., None])            # [S][nb][H]
    old = scale_of[slot]
    held = (off > 0)[:, None, None] & (torch.arange(nb, device=x.device) == 0)[None, :, None]
    held = held & (old > 0)
    ma, ea = torch.frexp(amax)
    ml, el = torch.frexp(old * FITS[kind])
    up = torch.where(held & (amax > 0), (ea - el + (ma > ml)).clamp(min=0), torch.zeros_like(ea))
    s = torch.where(held, old * _pow2(up), _quotient(amax, kind))
    scale_of.index_put_((slot,), torch.where(touched[..., None], s, old))
    # the rows that the first block held already
    r = ((pg[:, 0, None, None] * H + torch.arange(H, device=x.device)[None, :, None]) * page
         + ((first[:, 0] % per_page) * T)[:, None, None] + torch.arange(T, device=x.device))
    was = row_of[r].view(store.dtype)
    less = _codes(_values(was) * _pow2(-up[:, 0, :, None, None]), kind)
    keep = (torch.arange(T, device=x.device)[None, :] >= off[:, None])[:, None, :, None]
    row_of.index_put_((r,), torch.where(keep, _bytes(was), _bytes(less)))
    # the new rows
    sx = s.gather(1, (at // T)[..., None].expand(S, n, H))[..., None]
    y = _codes(torch.where(sx > 0, x / sx, torch.zeros_like(x)), kind)
    tok = pos[:, None] + torch.arange(n, device=x.device)[None, :]
    pt = table.long().gather(1, tok // page)
    r = ((pt[..., None] * H + torch.arange(H, device=x.device)) * page + (tok % page)[..., None])
    row_of.index_put_((r,), _bytes(y))


def _decode(st):
    c = st["case"]
    q, table, lens = st["q"], st["table"].long().clamp(min=0), st["lens"].long()
    B, Q, Hq, H, D, page, T = (c["batch"], c["q_len"], c["heads"], c["heads_kv"], c["head_dim"],
                               c["page"], c["block"])
    n = table.shape[1] * page
    pos = torch.arange(n, device=q.device)

    def gathered(store, scales):
        x = _values(_bytes(store[0])[table].view(store.dtype))       # [B][pages][H][page][D]
        x = x.reshape(B, -1, H, page // T, T, D) * scales[0][table][..., None, None]
        return x.reshape(B, -1, H, page, D).transpose(1, 2).reshape(B, H, n, D)

    last = lens[:, None] - Q + torch.arange(Q, device=q.device)[None, :]     # [B][Q]
    seen = (pos <= last[..., None]) & (pos < lens[:, None, None])
    if c["window"]:
        seen &= pos > last[..., None] - c["window"]
    seen = seen[:, None, :, None, :]                                         # [B][1][Q][1][n]
    x = q.float().reshape(B, Q, H, Hq // H, D).transpose(1, 2).reshape(B, H, -1, D)
    s = (x / math.sqrt(D)) @ gathered(st["k"], st["ks"]).transpose(2, 3)
    s = s.reshape(B, H, Q, Hq // H, n).masked_fill(~seen, -math.inf)
    m = s.amax(dim=-1, keepdim=True)
    p = torch.exp(s - torch.where(m > -math.inf, m, torch.zeros_like(m)))
    l = p.sum(dim=-1, keepdim=True)
    v = gathered(st["v"], st["vs"])
    v = v.masked_fill((pos[None, :] >= lens[:, None])[:, None, :, None], 0.0)
    o = (p / torch.where(l > 0, l, torch.ones_like(l))).reshape(B, H, -1, n) @ v
    o = o.reshape(B, H, Q, Hq // H, D).transpose(1, 2).reshape(B, Q, Hq, D)
    return o if Q > 1 else o[:, 0]


def _move(st, src, dst):
    for t in (st["k"], st["ks"], st["v"], st["vs"]):
        b = _bytes(t)
        b[:, dst] = b[:, src]


def _give_back(refs, table, taken):
    refs.scatter_add_(0, table.clamp(min=0)[taken >= 0].reshape(-1).long(),
                      -(taken >= 0).int()[taken >= 0].reshape(-1))


def _free_ids(refs):
    """Page ids, the free ones first in ascending order, and how many are free."""
    free = refs == 0
    return torch.sort((~free).int(), stable=True).indices, free.sum()


def _fork(st):
    page, refs, table, lens = st["case"]["page"], st["refs"], st["table"], st["lens"]
    par, ch = st["parents"].long(), st["children"].long()
    p = torch.arange(table.shape[1], device=table.device)
    n = lens[par].long()
    full = n // page
    shared = torch.where(p < full[:, None], table[par], -1)
    refs.scatter_add_(0, shared.clamp(min=0).reshape(-1).long(), (shared >= 0).int().reshape(-1))
    old = table[ch]
    refs.scatter_add_(0, old.clamp(min=0).reshape(-1).long(), -(old >= 0).int().reshape(-1))
    part = n % page > 0
    ids, _ = _free_ids(refs)
    fresh = ids[(torch.cumsum(part, 0) - 1).clamp(min=0)].int()
    at = full.clamp(max=table.shape[1] - 1)
    src = table[par, at]
    dst = torch.where(part, fresh, src)
    refs.scatter_add_(0, fresh.long(), part.int())
    shared.scatter_(1, at[:, None], torch.where(part, fresh, shared.gather(1, at[:, None])[:, 0])
                    [:, None])
    table[ch] = shared
    lens[ch] = lens[par]
    _move(st, src.clamp(min=0).long(), dst.clamp(min=0).long())


def _resize(st):
    page, refs, table, lens = st["case"]["page"], st["refs"], st["table"], st["lens"]
    p = torch.arange(table.shape[1], device=table.device)
    want = p < ((lens + page - 1) // page)[:, None]
    gone = ~want & (table >= 0)
    refs.scatter_add_(0, table.clamp(min=0).reshape(-1).long(), -gone.int().reshape(-1))
    table.masked_fill_(gone, -1)
    missing = want & (table < 0)
    ids, n_free = _free_ids(refs)
    rank = torch.cumsum(missing.reshape(-1), 0).reshape(table.shape) - 1
    got = missing & (rank < n_free)
    fresh = ids[rank.clamp(min=0, max=ids.numel() - 1)].int()
    table.copy_(torch.where(got, fresh, table))
    refs.scatter_add_(0, fresh.reshape(-1).long(), got.int().reshape(-1))


def _compact(st):
    refs, table = st["refs"], st["table"]
    ids = torch.arange(refs.numel(), device=refs.device)
    used = refs > 0
    n = used.sum()
    src = (used & (ids >= n)).nonzero()[:, 0]
    dst = (~used & (ids < n)).nonzero()[:, 0]
    to = ids.int()
    to[src] = dst.int()
    st["table_out"].copy_(torch.where(table >= 0, to[table.clamp(min=0).long()], table))
    st["refs_out"].zero_()
    st["refs_out"].scatter_add_(0, to.long(), refs)
    st["n_used"].copy_(n.int().reshape(1))
    _move(st, src, dst)


# ---- one pass --------------------------------------------------------------

def run(st):
    c = st["case"]
    op = c["op"]
    cache = dict(k=st["k"], ks=st["ks"], v=st["v"], vs=st["vs"])
    if own:
        from int8_kv_cache_02_gb300 import binding
    if op == "append":
        if own:
            binding.kv_quant_append(st["pool"], 0, st["k_new"], st["v_new"], st["pos"], st["table"])
        else:
            _append_one(st["k"], st["ks"], st["k_new"], st["pos"], st["table"], c)
            _append_one(st["v"], st["vs"], st["v_new"], st["pos"], st["table"], c)
        return cache
    if op == "decode":
        if not own:
            if c["append"]:
                at = st["lens"] - 1
                _append_one(st["k"], st["ks"], st["k_new"][:, None], at, st["table"], c)
                _append_one(st["v"], st["vs"], st["v_new"][:, None], at, st["table"], c)
            out = _decode(st)
        elif c["q_len"] > 1:
            out = st["out"]
            binding.attn_decode_multi_int8(st["pool"], 0, st["q"], st["lens"], st["table"], out,
                                           st["workspace"], n_splits=st["splits"])
        elif c["append"]:
            out = st["out"]
            binding.attn_decode_append_int8(st["pool"], 0, st["q"], st["k_new"], st["v_new"],
                                            st["lens"], st["table"], out, st["workspace"],
                                            window=c["window"], n_splits=st["splits"])
        else:
            out = st["out"]
            binding.attn_decode_int8(st["pool"], 0, st["q"], st["lens"], st["table"], out,
                                     st["workspace"], window=c["window"], n_splits=st["splits"])
        return dict(out=out, **cache) if c["append"] else dict(out=out)
    if op == "copy":
        if own:
            binding.kv_pages_copy(st["pool"], st["src"], st["dst"])
        else:
            _move(st, st["src"].long(), st["dst"].long())
        return cache
    if op == "fork":
        if own:
            binding.kv_pages_fork(st["pool"], st["refs"], st["table"], st["lens"], st["parents"],
                                  st["children"], st["workspace"])
        else:
            _fork(st)
        return dict(refs=st["refs"], table=st["table"], lens=st["lens"], **cache)
    if op == "resize":
        if own:
            binding.kv_pages_resize(st["pool"], st["refs"], st["table"], st["lens"],
                                    st["workspace"])
        else:
            _resize(st)
        return dict(refs=st["refs"], table=st["table"])
    if own:
        binding.kv_pages_compact(st["pool"], st["refs"], st["table"], st["refs_out"],
                                 st["table_out"], st["n_used"], st["workspace"])
    else:
        _compact(st)
    return dict(refs=st["refs_out"], table=st["table_out"], n_used=st["n_used"], **cache)


# ---- what a pass cannot do without -----------------------------------------

def work(case):
    c = case
    page, T = c["page"], c["block"]
    row = 2 * c["heads_kv"] * c["head_dim"]                 # K and V codes of one token
    page_bytes = page * row + 2 * c["heads_kv"] * (page // T) * 4
    op = c["op"]
    if op == "append":
        n = c["seqs"] * c["n_new"]
        return {"bytes": 3 * n * row + 8 * c["heads_kv"] * (n / T + c["seqs"])
                + 4 * c["seqs"] * (1 + -(-c["n_new"] // page)), "flops": 4 * n * row}
    if op == "decode":
        n = (c["min_len"] + c["max_len"]) / 2          # the seed decides: their mean
        if c["window"]:
            n = min(n, c["window"])
        live = c["batch"] - (c["empty"] if c["batch"] > c["empty"] else 0)
        tokens = live * n
        io = c["batch"] * c["q_len"] * c["heads"] * c["head_dim"] * (2 + 4)
        return {"bytes": tokens * (row + 8 * c["heads_kv"] / T + 4 / page) + io + 4 * c["batch"]
                + (3 * c["batch"] * row if c["append"] else 0),
                "flops": 4 * tokens * c["q_len"] * c["heads"] * c["head_dim"] + 1}
    L = c["layers"]
    if op == "copy":
        return {"bytes": c["copies"] * (2 * L * page_bytes + 8), "flops": 0}
    mean = max(1, c["max_len"] / 2)
    if op == "fork":
        n = c["parents"] * c["per_parent"]
        return {"bytes": n * (2 * L * page_bytes + 4 * (4 + 3 * mean / page)) + 4 * c["n_pages"],
                "flops": 0}
    entries = c["rows"] * -(-(c["max_len"] + 1) // page)
    if op == "resize":
        return {"bytes": 4 * (entries * 1.5 + c["n_pages"] * 1.25 + c["rows"]), "flops": 0}
    used = min(c["n_pages"], c["rows"] * (mean / page + 0.5))
    moved = used * (1 - used / c["n_pages"])
    return {"bytes": moved * 2 * L * page_bytes + 8 * (entries + c["n_pages"]), "flops": 0}


# ---- the definitions in 64 bits --------------------------------------------

def _exact_append(codes, scales, x, pos, table, c):
    """One store [pages][heads][page][head_dim] in 64 bits (values in units of the scale) and its
    scales [pages][heads][blocks], block by block.  A code is decided on the quotient rounded to
    32 bits, as the operator defines it."""
    T, page, kind = c["block"], c["page"], c["kind"]
    pos, table = pos.tolist(), table.tolist()

    def rounded(y):
        y = y.float()
        return (torch.clamp(torch.round(y), -127, 127) if kind == "int8"
                else torch.clamp(y, -448, 448).to(torch.float8_e4m3fn)).double()

    for b in range(x.shape[0]):
        i = 0
        while i < x.shape[1]:
            p = pos[b] + i
            n = min(T - p % T, x.shape[1] - i)
            new = x[b, i:i + n].double().transpose(0, 1)                    # [heads][n][head_dim]
            top = new.abs().amax(dim=(1, 2))
            pg, r0, blk, at = table[b][p // page], p % T, (p % page) // T, p % page
            s = (top / QMAX[kind]).float().double()
            if r0:
                was = scales[pg, :, blk]
                grown = was.clone()
                limit = (was * FITS[kind]).float().double()
                for _ in range(64):
                    more = (top > limit) & (was > 0)
                    grown, limit = torch.where(more, 2 * grown, grown), torch.where(more, 2 * limit,
                                                                                    limit)
                grown = torch.where(was > 0, grown, s)
                ratio = torch.where(was > 0, was / grown, torch.ones_like(was))
                lo = at - r0
                codes[pg, :, lo:at] = rounded(codes[pg, :, lo:at] * ratio[:, None, None])
                s = grown
            scales[pg, :, blk] = s
            y = torch.where(s[:, None, None] > 0, new / s[:, None, None], torch.zeros_like(new))
            codes[pg, :, at:at + n] = rounded(y)
            i += n


def _exact_decode(st, k, ks, v, vs):
    c = st["case"]
    T, page, G, Q = c["block"], c["page"], c["heads"] // c["heads_kv"], c["q_len"]
    q = st["q"].double().reshape(c["batch"], Q, c["heads"], -1)
    out = torch.zeros_like(q)
    for b, n in enumerate(st["lens"].tolist()):
        if not n:
            continue
        ids = st["table"][b, :-(-n // page)].long()
        rows = []
        for codes, scales in ((k, ks), (v, vs)):
            x = codes[ids].double() if codes.dtype == torch.float64 else \
                _bytes(codes)[ids].view(codes.dtype).float().double()
            x = x * scales[ids].double().repeat_interleave(T, dim=2)[..., None]
            rows.append(x.permute(1, 0, 2, 3).reshape(c["heads_kv"], -1, c["head_dim"])[:, :n])
        for i in range(Q):
            last = n - Q + i
            if last < 0:
                continue
            a = max(0, last + 1 - c["window"]) if c["window"] else 0
            for h in range(c["heads_kv"]):
                s = q[b, i, h * G:(h + 1) * G] @ rows[0][h, a:last + 1].T / math.sqrt(c["head_dim"])
                out[b, i, h * G:(h + 1) * G] = torch.softmax(s, dim=1) @ rows[1][h, a:last + 1]
    return out if Q > 1 else out[:, 0]


def _exact_pages(st):
    """The moved scales, with the pages handled one by one on the host."""
    c = st["case"]
    page, moves = c["page"], []
    if c["op"] == "copy":
        moves = list(zip(st["src"].tolist(), st["dst"].tolist()))
    else:
        refs, table, lens = st["refs"].tolist(), st["table"].tolist(), st["lens"].tolist()
    if c["op"] == "fork":
        pairs = list(zip(st["parents"].tolist(), st["children"].tolist()))
        for a, b in pairs:
            for i in range(lens[a] // page):
                refs[table[a][i]] += 1
        for a, b in pairs:
            for e in table[b]:
                if e >= 0:
                    refs[e] -= 1
        free = iter([i for i, r in enumerate(refs) if r == 0])
        moves = [(table[a][lens[a] // page], next(free)) for a, b in pairs if lens[a] % page]
    if c["op"] == "compact":
        n = sum(r > 0 for r in refs)
        moves = list(zip([i for i in range(n, len(refs)) if refs[i]],
                         [i for i in range(n) if not refs[i]]))
    out = {}
    for name in ("ks", "vs"):
        x = st[name].double().clone()
        for a, b in moves:
            x[:, b] = st[name][:, a].double()
        out[name] = x
    return out


def exact(case, seed):
    c = dict(case)
    if c["op"] == "resize":
        return None                       # whole numbers only
    st = prepare(c, seed)
    if c["op"] in ("copy", "fork", "compact"):
        return _exact_pages(st)
    res = {}
    k, ks, v, vs = st["k"][0], st["ks"][0], st["v"][0], st["vs"][0]
    if c["op"] == "append" or c["append"]:
        single = c["op"] == "decode"
        pos = st["lens"] - 1 if single else st["pos"]
        made = []
        for codes, scales, x in ((k, ks, st["k_new"]), (v, vs, st["v_new"])):
            codes, scales = codes.float().double(), scales.double()
            _exact_append(codes, scales, x[:, None] if single else x, pos, st["table"], c)
            made += [codes, scales]
        k, ks, v, vs = made
        res = dict(k=k[None] if c["kind"] == "e4m3" else None, ks=ks[None],
                   v=v[None] if c["kind"] == "e4m3" else None, vs=vs[None])
    if c["op"] == "decode":
        res["out"] = _exact_decode(st, k, ks, v, vs)
    return res
