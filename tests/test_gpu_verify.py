"""Verification of drafted tokens on the GPU: whole numbers, equal to the oracle's."""

import numpy as np
import pytest
import torch

from oracle import verify

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from int8_kv_cache_02_gb300 import build
    build.build()


def _case(g, B, n, V, sharp=3.0, drafts=True):
    logits = sharp * torch.randn((B, n + 1, V), generator=g)
    target = torch.softmax(logits, dim=2)
    near = logits[:, :n] + torch.randn((B, n, V), generator=g)
    draft = torch.softmax(near, dim=2)
    x = (torch.multinomial(draft.reshape(-1, V), 1, generator=g).reshape(B, n) if n else
         torch.zeros((B, 0), dtype=torch.long)).int()
    return (target, draft if drafts else None, x, torch.rand((B, n), generator=g),
            torch.rand((B,), generator=g))


def _call(target, draft, x, u, s, n_drafts=None, lens=None, in_place=False):
    from int8_kv_cache_02_gb300 import binding
    B, n = x.shape
    tokens = torch.full((B, n + 1), -7, dtype=torch.int32, device="cuda")
    acc = torch.full((B,), -7, dtype=torch.int32, device="cuda")

    def up(t):
        return None if t is None else (t if t.is_cuda else t.cuda())
    before = None if lens is None else torch.tensor(lens, dtype=torch.int32, device="cuda")
    after = before if in_place or before is None else torch.empty_like(before)
    binding.kv_verify_drafts(up(target), up(x), up(u), up(s), tokens, acc, draft_probs=up(draft),
                             n_drafts=None if n_drafts is None else
                             torch.tensor(n_drafts, dtype=torch.int32, device="cuda"),
                             seq_lens=before, seq_lens_out=after)
    torch.cuda.synchronize()
    return tokens.cpu().numpy(), acc.cpu().numpy(), None if after is None else after.cpu().numpy()


def _check(target, draft, x, u, s, **kw):
    got = _call(target, draft, x, u, s, **kw)
    want = verify.batch(target.cpu().numpy(), None if draft is None else draft.cpu().numpy(),
                        x.cpu().numpy(), u.cpu().numpy(), s.cpu().numpy(), kw.get("n_drafts"),
                        kw.get("lens"))
    for a, b in zip(got, want):
        assert a is None and b is None or np.array_equal(a, b), (a, b)
    return got


@pytest.mark.parametrize("V", [1, 2, 31, 33, 255, 4096, 4097, 32000, 50001])
@pytest.mark.parametrize("n", [0, 1, 4])
@pytest.mark.parametrize("drafts", [True, False])
def test_vocabularies(V, n, drafts):
    g = torch.Generator().manual_seed(V + n)
    _check(*_case(g, 5, n, V, drafts=drafts), lens=[100, 7, 8, 9, 1000])


@pytest.mark.parametrize("n", [31, 32, 33, 63, 200])
def test_long_drafts(n):
    """Likely drafts, so that refusals come late; several rounds of 32."""
    g = torch.Generator().manual_seed(n)
    target, draft, x, u, s = _case(g, 6, n, 40, sharp=1.0)
    draft[1:] = target[1:, :n]
    for b in range(1, 6):
        x[b] = torch.multinomial(draft[b], 1, generator=g)[:, 0].int()
    u[3, n - 1] = 1.0
    u[4, min(n - 1, 40)] = float("nan")
    got = _check(target, draft, x, u, s)
    assert got[1][1] == n and got[1][3] == n - 1 and got[1][4] == min(n - 1, 40)


def test_ragged_sequences():
    """None, some, all, more than there are, and sequences that take no part."""
    g = torch.Generator().manual_seed(3)
    for drafts in (True, False):
        _check(*_case(g, 7, 5, 700, drafts=drafts), n_drafts=[5, 0, 3, -1, 9, 1, -2147483648],
               lens=[50] * 7, in_place=True)


def test_numbers_at_their_ends():
    """Random numbers of 0, just below 1, 1 and more; weights at both ends of a row."""
    V = 5000
    for where in ([0], [V - 1], [0, V - 1], [2048], [639, 640]):
        p = torch.zeros((6, 1, V))
        p[:, :, where] = 1.0 / len(where)
        s = torch.tensor([0.0, 0.5, 1.0 - 2.0 ** -24, 1.0, 7.0, float("nan")])
        x = torch.zeros((6, 0), dtype=torch.int32)
        got = _check(p, None, x, torch.zeros((6, 0)), s)
        assert set(got[0][:, 0].tolist()) <= set(where) and got[0][0, 0] == where[0]


def test_rows_with_nothing_left():
    """p = q, rows of zeros, NaN, infinities and negative values, drafts that are no tokens."""
    g = torch.Generator().manual_seed(4)
    target, draft, x, u, s = _case(g, 8, 2, 600)
    u[:] = 0.999
    draft[0] = target[0, :2]            # taken: u < 1
    draft[1, 0] = target[1, 0]
    x[1, 0] = 3
    u[1, 0] = 1.0                       # refused, and nothing is left: by p itself
    target[2] = 0.0
    target[3] = float("nan")
    target[4, 0, 5:9] = float("inf")
    target[5, 0, ::2] = -0.5
    x[6] = torch.tensor([600, 1])
    x[7] = torch.tensor([-1, 1])
    for d in (draft, None):
        got = _check(target, d, x, u, s)
        assert got[0][2, 0] == -1 and got[0][3, 0] == -1 and got[1][6] == 0 and got[1][7] == 0


def test_small_probabilities_are_whole_units():
    """Values around 2^-37, 2^-60 and below, and subnormal ones."""
    V = 400
    p = torch.zeros((3, 1, V))
    p[:, 0, :] = torch.tensor([2.0 ** -e for e in range(20, 148)] + [0.0] * (V - 128))
    p[1, 0, :40] = 0.0                    # below 2^-60 nothing counts
    p[2, 0, :36] = 0.0
    x = torch.zeros((3, 0), dtype=torch.int32)
    for s in (0.0, 0.3, 0.9, 0.9999):
        _check(p, None, x, torch.zeros((3, 0)), torch.full((3,), s))


def test_padded_rows_and_the_same_token_twice():
    """A slice of wider rows; drafts that repeat a token; a batch of one."""
    g = torch.Generator().manual_seed(6)
    target, draft, x, u, s = _case(g, 4, 3, 1001)
    wide = torch.full((4, 4, 1100), 9.0, device="cuda")
    wide[..., :1001] = target.cuda()
    x[:] = x[:, :1]
    a = _check(wide[..., :1001], draft, x, u, s)
    b = _check(target, draft, x, u, s)
    assert np.array_equal(a[0], b[0])
    _check(target[:1], draft[:1], x[:1], u[:1], s[:1])


def test_the_batch_does_not_matter():
    """A sequence's result is the same alone and among others; large vocabularies."""
    g = torch.Generator().manual_seed(7)
    c = _case(g, 40, 2, 131072)
    whole = _check(*c)
    for b in (0, 17, 39):
        alone = _call(*(t[b:b + 1] for t in c))
        assert np.array_equal(alone[0], whole[0][b:b + 1])


def test_replayed_on_another_stream():
    from int8_kv_cache_02_gb300 import binding
    g = torch.Generator().manual_seed(8)
    first = [t.cuda() for t in _case(g, 3, 4, 3000)]
    tokens = torch.empty((3, 5), dtype=torch.int32, device="cuda")
    acc, lens = (torch.zeros(3, dtype=torch.int32, device="cuda") for _ in range(2))
    target, draft, x, u, s = first
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(stream):
        with torch.cuda.graph(graph, stream=stream):
            binding.kv_verify_drafts(target, x, u, s, tokens, acc, draft_probs=draft, seq_lens=lens,
                                     seq_lens_out=lens)
        total = np.zeros(3, np.int64)
        for _ in range(5):
            new = _case(g, 3, 4, 3000)
            for t, h in zip(first, new):
                t.copy_(h)
            graph.replay()
            stream.synchronize()
            want = verify.batch(*(t.numpy() for t in new))
            assert np.array_equal(tokens.cpu().numpy(), want[0])
            assert np.array_equal(acc.cpu().numpy(), want[1])
            total -= 4 - want[1]
            assert np.array_equal(lens.cpu().numpy(), total)


def test_rows_that_are_no_probabilities():
    """Sums of 16 and more: some value of the vocabulary, or -1; the drafts before it stand."""
    for V in (40, 5000, 33001):
        p = torch.ones((3, 2, V))
        p[1] *= 0.01
        x = torch.zeros((3, 1), dtype=torch.int32)
        for n in (None, [0, 0, 0]):
            got = _call(p, None, x, torch.full((3, 1), 0.5), torch.rand(3), n_drafts=n)
            assert ((got[0] >= -1) & (got[0] < V)).all()
            assert got[1].tolist() == ([1, 0, 1] if n is None else [0, 0, 0])


def test_every_exponent_is_exact():
    """Values of random mantissas at every exponent, alone in their rows and against another's."""
    g = torch.Generator().manual_seed(13)
    V, B = 64, 140
    p = torch.zeros((B, 2, V))
    e = torch.arange(B).float()[:, None]
    p[:, 0] = (1 + torch.rand((B, V), generator=g)) * 2.0 ** (-1 - e) / V
    p[:, 1] = (1 + torch.rand((B, V), generator=g)) * 2.0 ** (-1 - e) / V
    q = (1 + torch.rand((B, 1, V), generator=g)) * 2.0 ** (-1 - e[..., None]) / V
    x = torch.randint(0, V, (B, 1), generator=g, dtype=torch.int32)
    for u in (0.0, 1.0):
        _check(p, q, x, torch.full((B, 1), u), torch.rand(B, generator=g))


def test_drafts_of_no_probability():
    """The drafted token's own entries outside [0, 1] and NaN, in either row: they count as the nearest
    of the two, NaN as 0.  Each pair's verdict is written out, not the oracle's alone."""
    inf, nan = float("inf"), float("nan")
    #        p, q, u, taken: u q < p with both in [0, 1]
    rows = [(1.0, 3.0, 0.9, 1), (1.0, inf, 0.999, 1), (0.5, 3.0, 0.4, 1), (0.5, 3.0, 0.5, 0),
            (0.0, -0.5, 0.5, 0), (-0.5, -1.0, 0.9, 0), (nan, -1.0, 0.9, 0), (0.25, nan, 0.999, 1),
            (0.0, nan, 0.5, 0), (nan, 0.5, 0.0, 0), (nan, nan, 0.0, 0), (7.0, 1.0, 0.999, 1),
            (inf, inf, 0.999, 1), (-inf, -inf, 0.5, 0), (2.0 ** -140, -1.0, 0.9, 1),
            (2.0 ** -149, 0.0, 0.5, 1), (0.0, 0.0, 0.0, 0)]
    B, V, at = len(rows), 70, 37
    g = torch.Generator().manual_seed(15)
    target = torch.rand((B, 2, V), generator=g) / V
    draft = torch.rand((B, 1, V), generator=g) / V
    x = torch.full((B, 1), at, dtype=torch.int32)
    u = torch.zeros((B, 1))
    for b, (p, q, r, _) in enumerate(rows):
        target[b, 0, at], draft[b, 0, at], u[b, 0] = p, q, r
    got = _check(target, draft, x, u, torch.rand(B, generator=g))
    assert got[1].tolist() == [r[3] for r in rows]
    got = _check(target, None, x, u, torch.rand(B, generator=g))        # (q is 1)
    assert got[1].tolist() == [int(r[2] < min(max(r[0], 0.0), 1.0)) if r[0] == r[0] else 0 for r in rows]
