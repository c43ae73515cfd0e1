"""Page calls on the GPU against the sequential oracle; whole pools byte for byte."""

import random

import numpy as np
import pytest
import torch

from oracle import pages as opages
from tests import block_util as bu

pytestmark = pytest.mark.gpu

POOLS = [("k8v8", 2, 2, 64, 64, 16), ("k16v8", 1, 3, 128, 64, 32), ("q4_0", 3, 1, 64, 64, 16),
         ("k8v8_block", 2, 1, 64, 16, 16), ("f8_block", 1, 5, 256, 32, 128),
         ("k8v8_block", 2, 3, 64, 16, 32)]


def _pool(spec, n_pages, seed=0):
    from int8_kv_cache_02_gb300 import binding, build
    build.build()
    variant, layers, Hkv, D, gs, ps = spec
    p = binding.KVPool(layers, Hkv, D, gs, ps, n_pages, variant)
    g = torch.Generator(device="cuda").manual_seed(seed)
    for t in _regions(p):
        t.copy_(torch.randint(0, 256, t.shape, generator=g, device="cuda", dtype=torch.uint8))
    return p


def _regions(p):
    return [t.view(torch.uint8) for t in (p.k_store, p.v_store, p.k_scales, p.v_scales)
            if t is not None]


def _snapshot(p):
    return [t.cpu() for t in _regions(p)]


def _assert_moved(p, before, moves, what=""):
    for t, was in zip(_regions(p), before):
        want = was.clone()
        for a, b in moves:
            want[:, b] = was[:, a]
        assert torch.equal(t.cpu(), want), what


def _dev(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("spec", POOLS)
def test_copy(spec):
    from int8_kv_cache_02_gb300 import binding as b
    p = _pool(spec, 11)
    before = _snapshot(p)
    b.kv_pages_copy(p, _dev([3, 0, -1, 5, 7, 3]), _dev([1, 2, 4, -1, 7, 9]))
    _assert_moved(p, before, [(3, 1), (0, 2), (3, 9)])
    assert b.kv_pool_read_device_error(p) == 0
    before = _snapshot(p)
    b.kv_pages_copy(p, _dev([11, 0, 2]), _dev([1, 99, 10]))
    _assert_moved(p, before, [(2, 10)])
    assert b.kv_pool_read_device_error(p) == b.DEVERR_PAGE_ID
    b.kv_pages_copy(p, _dev([]), _dev([]))


def test_copy_of_many_pages_and_odd_chunks():
    """Pages of several copy chunks, the last one partial; more chunks than blocks run at once."""
    from int8_kv_cache_02_gb300 import binding as b
    p = _pool(("f8_block", 2, 5, 256, 64, 64), 301)
    before = _snapshot(p)
    ids = torch.randperm(301, generator=torch.Generator().manual_seed(0)).int()
    b.kv_pages_copy(p, ids[:150].cuda(), ids[150:300].contiguous().cuda())
    _assert_moved(p, before, list(zip(ids[:150].tolist(), ids[150:300].tolist())))


def _codes(errors):
    from int8_kv_cache_02_gb300 import binding as b
    names = dict(page=b.DEVERR_PAGE_ID, length=b.DEVERR_LENGTH, no_page=b.DEVERR_NO_PAGE,
                 fork=b.DEVERR_FORK)
    return sum(names[e] for e in errors)


class _State:
    def __init__(self, spec, n_pages, rows, width):
        self.p, self.rows, self.width = _pool(spec, n_pages), rows, width
        self.refs, self.lens = [0] * n_pages, [0] * rows
        self.table = [[-1] * width for _ in range(rows)]
        self.d = dict(refs=_dev(self.refs), table=_dev(self.table), lens=_dev(self.lens))
        self.ws = self.p.pages_workspace(rows)
        self.ws.fill_(0xA5)                    # any contents

    def push(self):
        for n in self.d:
            self.d[n].copy_(_dev(getattr(self, n)))

    def check(self, moves, errors, before, what):
        from int8_kv_cache_02_gb300 import binding as b
        for n in self.d:
            got = self.d[n].cpu().tolist()
            assert got == getattr(self, n), f"{what}: {n}"
        assert b.kv_pool_read_device_error(self.p) == _codes(errors), what
        _assert_moved(self.p, before, moves, what)


@pytest.mark.parametrize("seed", range(4))
def test_random_calls_against_the_oracle(seed):
    """Resizes, forks and compactions in any order, pools that run out of pages, rows cut back,
    lists with padding, repeated and impossible forks."""
    from int8_kv_cache_02_gb300 import binding as b
    rng = random.Random(seed)
    spec = POOLS[seed]
    ps = spec[5]
    s = _State(spec, rng.choice([7, 40, 150]), rng.randint(2, 20), rng.randint(1, 12))
    for step in range(25):
        before = _snapshot(s.p)
        op = rng.choice(["resize", "resize", "fork", "compact"])
        if op == "resize":
            s.lens = [rng.choice([0, n, n + 1, rng.randint(0, s.width * ps + 3)]) for n in s.lens]
            s.d["lens"].copy_(_dev(s.lens))
            moves, err = opages.resize(s.refs, s.table, s.lens, ps)
            b.kv_pages_resize(s.p, s.d["refs"], s.d["table"], s.d["lens"], s.ws)
        elif op == "fork":
            n = rng.randint(1, s.rows)
            par = [rng.randint(-1, s.rows) for _ in range(n)]
            ch = [rng.randint(-1, s.rows) for _ in range(n)]
            moves, err = opages.fork(s.refs, s.table, s.lens, par, ch, ps)
            b.kv_pages_fork(s.p, s.d["refs"], s.d["table"], s.d["lens"], _dev(par), _dev(ch), s.ws)
        else:
            moves, err, used = opages.compact(s.refs, s.table)
            u = _dev([-7])
            if rng.random() < 0.5:             # in place
                b.kv_pages_compact(s.p, s.d["refs"], s.d["table"], s.d["refs"], s.d["table"], u,
                                   s.ws)
            else:
                r, t = torch.full_like(s.d["refs"], -3), torch.full_like(s.d["table"], -3)
                b.kv_pages_compact(s.p, s.d["refs"], s.d["table"], r, t, u, s.ws)
                s.d["refs"], s.d["table"] = r, t
            assert u.item() == used
        s.check(moves, err, before, f"seed {seed} step {step} {op}")


def test_bad_entries_and_counts():
    """Entries beyond the pool, counts that are too low already, entries of free pages."""
    from int8_kv_cache_02_gb300 import binding as b
    s = _State(POOLS[3], 6, 3, 3)
    s.refs, s.table, s.lens = [1, 0, 1, 2, 0, 0], [[0, 3, 99], [1, 3, -4], [2, -1, 6]], [48, 0, 40]
    s.push()
    before = _snapshot(s.p)
    moves, err = opages.resize(s.refs, s.table, s.lens, 16)
    b.kv_pages_resize(s.p, s.d["refs"], s.d["table"], s.d["lens"], s.ws)
    assert err == {"page"}
    s.check(moves, err, before, "resize")
    s.refs, s.table, s.lens = [1, 0, 1, 2, 0, 1], [[0, 3, 99], [1, 77, 3], [2, -1, 6]], [36, 0, 20]
    s.push()
    moves, err = opages.fork(s.refs, s.table, s.lens, [0], [1], 16)
    b.kv_pages_fork(s.p, s.d["refs"], s.d["table"], s.d["lens"], _dev([0]), _dev([1]), s.ws)
    s.check(moves, err, before, "fork")
    s.refs, s.table = [0, 2, 0, 0, 1, 1], [[1, 1, 0], [4, 88, 5], [-1, -1, 3]]
    s.push()
    moves, err, used = opages.compact(s.refs, s.table)
    u = _dev([0])
    b.kv_pages_compact(s.p, s.d["refs"], s.d["table"], s.d["refs"], s.d["table"], u, s.ws)
    assert u.item() == used == 3 and err == {"page"}
    s.check(moves, err, before, "compact")


def test_large_tables():
    """More entries and pages than threads; shared prefixes; a pool that just suffices."""
    from int8_kv_cache_02_gb300 import binding as b
    rows, width, ps, n_pages = 150, 300, 16, 20011
    s = _State(("k8v8_block", 1, 1, 64, 16, 16), n_pages, rows, width)
    g = torch.Generator().manual_seed(5)
    for step in range(3):
        s.lens = torch.randint(0, width * ps + 1, (rows,), generator=g).tolist()
        s.lens[:50] = [0] * 50
        s.d["lens"].copy_(_dev(s.lens))
        before = _snapshot(s.p)
        moves, err = opages.resize(s.refs, s.table, s.lens, ps)
        b.kv_pages_resize(s.p, s.d["refs"], s.d["table"], s.d["lens"], s.ws)
        s.check(moves, err, before, "resize")
        par, ch = [50 + i % 7 for i in range(50)], list(range(50))
        moves, err = opages.fork(s.refs, s.table, s.lens, par, ch, ps)
        b.kv_pages_fork(s.p, s.d["refs"], s.d["table"], s.d["lens"], _dev(par), _dev(ch), s.ws)
        s.check(moves, err, before, "fork")
        before = _snapshot(s.p)
        moves, err, used = opages.compact(s.refs, s.table)
        u = _dev([0])
        b.kv_pages_compact(s.p, s.d["refs"], s.d["table"], s.d["refs"], s.d["table"], u, s.ws)
        s.check(moves, err, before, "compact")
        assert u.item() == used and not err


def test_a_fork_that_cannot_copy_changes_nothing():
    """More page copies than a launch counts: refused before the table and the counts change."""
    from int8_kv_cache_02_gb300 import binding as b
    layers, forks = 4096, 2 ** 18              # times two chunks a layer's page: 2^31
    p = b.KVPool(layers, 1, 64, 16, 16, 2, "k8v8_block")
    refs, lens = _dev([1, 0]), torch.zeros(forks, dtype=torch.int32, device="cuda")
    table = torch.full((forks, 1), -1, dtype=torch.int32, device="cuda")
    par, ch = (torch.full((forks,), -1, dtype=torch.int32, device="cuda") for _ in range(2))
    table[0], lens[0], par[0], ch[0] = 0, 5, 0, 1
    was = [t.clone() for t in (refs, table, lens)]
    ws = p.pages_workspace(forks)
    with pytest.raises(b.Int8KVError, match="-6"):
        b.kv_pages_fork(p, refs, table, lens, par, ch, ws)
    for t, x in zip((refs, table, lens), was):
        assert torch.equal(t, x)
    b.kv_pages_fork(p, refs, table, lens, par[:-1].contiguous(), ch[:-1].contiguous(), ws)
    assert refs.tolist() == [1, 1] and table[:3, 0].tolist() == [0, 1, -1] and lens[1] == 5


def test_lengths_far_below_zero_are_empty_rows():
    """The lowest lengths int32 has: their rows' pages go back, and the others get the lowest
    free ones."""
    from int8_kv_cache_02_gb300 import binding as b
    s = _State(POOLS[3], 12, 4, 4)
    s.refs[:5] = [1] * 5
    s.table = [[0, 1, 2, -1], [3, -1, -1, -1], [4, -1, -1, -1], [-1] * 4]
    s.lens = [-2 ** 31, 40, -2 ** 31 + 20, 64]
    s.push()
    before = _snapshot(s.p)
    moves, err = opages.resize(s.refs, s.table, s.lens, 16)
    b.kv_pages_resize(s.p, s.d["refs"], s.d["table"], s.d["lens"], s.ws)
    s.check(moves, err, before, "resize")
    assert s.table[1] == [3, 0, 1, -1] and not err


@pytest.mark.parametrize("rows", [4096, 4097, 9000])
def test_forks_in_tables_of_many_rows(rows):
    """Up to 4096 rows every block keeps its own marks; beyond, the cluster shares them in the
    workspace. Repeated children, children that are parents, rows outside the table, padding."""
    from int8_kv_cache_02_gb300 import binding as b
    ps, width = 16, 3
    rng = random.Random(rows)
    s = _State(("k8v8_block", 1, 1, 64, 16, 16), rows * 2, rows, width)
    s.lens = [rng.randint(0, width * ps) if rng.random() < 0.6 else 0 for _ in range(rows)]
    s.d["lens"].copy_(_dev(s.lens))
    before = _snapshot(s.p)
    moves, err = opages.resize(s.refs, s.table, s.lens, ps)
    b.kv_pages_resize(s.p, s.d["refs"], s.d["table"], s.d["lens"], s.ws)
    s.check(moves, err, before, "resize")
    for step in range(2):
        n = rng.randint(rows // 2, rows)
        par = [rng.randint(-1, rows) for _ in range(n)]
        ch = [rng.choice([rng.randint(-1, rows), rng.randint(rows - 40, rows - 1)]) for _ in range(n)]
        if step:                # few parents: most forks take place
            par = [rng.randrange(30) if p >= 0 else p for p in par]
        before = _snapshot(s.p)
        moves, err = opages.fork(s.refs, s.table, s.lens, par, ch, ps)
        assert moves and "fork" in err
        b.kv_pages_fork(s.p, s.d["refs"], s.d["table"], s.d["lens"], _dev(par), _dev(ch), s.ws)
        s.check(moves, err, before, f"fork {step}")


def test_free_pages_behind_the_first_span():
    """A pool of more than twice the 65,536 pages that are searched at a time: pages from the
    second and the third span, from all of them at once, and none left."""
    from int8_kv_cache_02_gb300 import binding as b
    rows, width, ps, n_pages = 76, 2000, 16, 132500
    s = _State(("k8v8_block", 1, 1, 64, 16, 16), n_pages, rows, width)
    full = width * ps
    before = _snapshot(s.p)

    def resize(what):
        s.d["lens"].copy_(_dev(s.lens))
        moves, err = opages.resize(s.refs, s.table, s.lens, ps)
        b.kv_pages_resize(s.p, s.d["refs"], s.d["table"], s.d["lens"], s.ws)
        s.check(moves, err, before, what)
        return err

    s.lens = [full] * 32 + [0] * 44                      # 64,000 pages
    resize("first")
    s.lens[32:36] = [full] * 3 + [55]                    # over the border to the second span
    resize("second")
    s.lens[:32] = [full - 16 * (i % 2) for i in range(32)]      # holes in the first
    s.lens[40:71] = [full - 7] * 31                      # all of the second, some of the third
    assert not resize("third")
    moves, err = opages.fork(s.refs, s.table, s.lens, [40, 41, 35], [71, 72, 73], ps)
    b.kv_pages_fork(s.p, s.d["refs"], s.d["table"], s.d["lens"], _dev([40, 41, 35]),
                    _dev([71, 72, 73]), s.ws)
    assert min(d for _, d in moves) >= 2 * 65536 and not err
    s.check(moves, err, before, "fork")
    before = _snapshot(s.p)
    s.lens[74] = full
    assert resize("none left") == {"no_page"}
    s.lens[:20] = [0] * 20
    resize("back")
    moves, err, used = opages.compact(s.refs, s.table)
    u = _dev([0])
    b.kv_pages_compact(s.p, s.d["refs"], s.d["table"], s.d["refs"], s.d["table"], u, s.ws)
    assert u.item() == used and not err
    s.check(moves, err, before, "compact")


def test_refusals():
    from int8_kv_cache_02_gb300 import binding as b
    s = _State(POOLS[3], 6, 3, 3)
    d, ws = s.d, s.ws
    small = torch.zeros(s.ws.numel() - 1, dtype=torch.uint8, device="cuda")
    with pytest.raises(b.Int8KVError, match="-8"):
        b.kv_pages_resize(s.p, d["refs"], d["table"], d["lens"], small)
    with pytest.raises(b.Int8KVError, match="-3"):
        b.kv_pages_resize(s.p, d["refs"], d["table"], d["lens"],
                          torch.zeros(s.ws.numel() + 1, dtype=torch.uint8, device="cuda")[1:])
    with pytest.raises(b.Int8KVError, match="-1"):
        b.kv_pages_fork(s.p, d["refs"], d["table"], d["lens"], _dev([0] * 4), _dev([1] * 4), ws)
    with pytest.raises(ValueError, match="page_refs"):
        b.kv_pages_resize(s.p, d["refs"][:5], d["table"], d["lens"], ws)
    with pytest.raises(ValueError, match="page_table_out"):
        b.kv_pages_compact(s.p, d["refs"], d["table"], d["refs"], d["table"][:2], d["lens"], ws)
    with pytest.raises(ValueError, match="contiguous"):
        b.kv_pages_copy(s.p, torch.zeros((4, 2), dtype=torch.int32, device="cuda")[:, 0],
                        d["refs"][:4])
    b.kv_pages_resize(s.p, d["refs"], d["table"][:0], d["lens"][:0], ws)


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
def test_a_served_batch_from_prompt_to_compaction(kind):
    """The calls as a server makes them: pages for prompts, append, decode; two beams forked off
    each; every sequence grows by its own tokens, through a captured step; some end; the pool is
    compacted; the others go on.  Every step's output against fp64 over an unpaged model."""
    from int8_kv_cache_02_gb300 import binding as b
    Hkv, G, D, gs, ps, rows, width = 2, 4, 64, 16, 32, 6, 6
    dev, _ = bu.make_pools(kind, Hkv, D, gs, ps, 24)
    refs, table = torch.zeros(24, dtype=torch.int32, device="cuda"), \
        torch.full((rows, width), -1, dtype=torch.int32, device="cuda")
    lens = torch.zeros(rows, dtype=torch.int32, device="cuda")
    ws, dws = dev.pages_workspace(rows), dev.decode_workspace(rows, Hkv * G, 4)
    g = torch.Generator().manual_seed(21)
    # one pool of the oracle's per row, with its own pages in order: no sharing, no paging
    own = bu.oblock.BlockPool(1, Hkv, D, gs, ps, rows * width, kind)
    place = np.arange(rows * width).reshape(rows, width)

    def rows_of(n, m):
        return (torch.randn((n, m, Hkv, D), generator=g).half(),
                torch.randn((n, m, Hkv, D), generator=g).half())

    prompt = [50, 64]
    lens[:2] = _dev(prompt)
    b.kv_pages_resize(dev, refs, table, lens, ws)
    for i, n in enumerate(prompt):
        k, v = rows_of(1, n)
        bu.append(dev, None, 0, k, v, [0], table[i:i + 1].cpu())
        own.append(0, k.numpy(), v.numpy(), [0], place[i:i + 1])
    b.kv_pages_fork(dev, refs, table, lens, _dev([0, 0, 1, 1]), _dev([2, 3, 4, 5]), ws)
    for p, c in ((0, 2), (0, 3), (1, 4), (1, 5)):
        for t in (own.k_store, own.v_store, own.k_scales, own.v_scales):
            t[0, place[c]] = t[0, place[p]]
    n = prompt + [50, 50, 64, 64]
    assert lens.tolist() == n and refs.sum().item() == 2 + 2 + 4 * 2

    q = torch.zeros((rows, Hkv * G, D), dtype=torch.float16, device="cuda")
    k1, v1 = (torch.zeros((rows, Hkv, D), dtype=torch.float16, device="cuda") for _ in range(2))
    out = torch.empty((rows, Hkv * G, D), device="cuda")
    live = torch.ones(rows, dtype=torch.int32, device="cuda")

    def step():
        lens.add_(live)
        b.kv_pages_resize(dev, refs, table, lens, ws)
        b.attn_decode_append_int8(dev, 0, q, k1, v1, lens, table, out, dws, n_splits=4)

    saved = lens.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    assert torch.equal(saved, lens)            # capturing ran nothing
    used = _dev([0])
    for s in range(24):
        if s == 12:                            # rows 1 and 3 end; the pool is compacted
            for i in (1, 3):
                live[i] = 0
                lens[i] = n[i] = 0
            b.kv_pages_resize(dev, refs, table, lens, ws)
            b.kv_pages_compact(dev, refs, table, refs, table, used, ws)
            assert used.item() == (refs > 0).sum().item() == (refs[:used.item()] > 0).sum().item()
        k, v = rows_of(rows, 1)
        k = (k * (1 + s)).half()               # blocks grow now and then
        qs = torch.randn((rows, 1, Hkv * G, D), generator=g).half()
        q.copy_(qs[:, 0])
        k1.copy_(k[:, 0])
        v1.copy_(v[:, 0])
        graph.replay()
        for i in range(rows):
            if n[i]:
                own.append(0, k[i:i + 1].numpy(), v[i:i + 1].numpy(), [n[i]], place[i:i + 1])
                n[i] += 1
        assert lens.tolist() == n
        ref = bu.reference(own, 0, qs, n, torch.from_numpy(place))
        bu.assert_close(out.cpu().numpy(), ref[:, 0], z_max=128, what=f"step {s}")
    counts = torch.bincount(table[table >= 0].long(), minlength=24)
    assert torch.equal(counts.int(), refs)
    err = b.kv_pool_read_device_error(dev)
    assert err == b.DEVERR_LENGTH              # (the fused append of an ended row has no place)
