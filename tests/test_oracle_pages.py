"""The page-table oracle pinned by hand-made cases and invariants (CPU only)."""

import random

from oracle import pages


def _counts(refs, table):
    n = [0] * len(refs)
    for row in table:
        for e in row:
            if e >= 0:
                n[e] += 1
    return n


def test_resize_by_hand():
    refs, table = [1, 0, 1, 1, 0], [[3, 0, -1], [2, -1, -1], [-1, -1, -1]]
    moves, err = pages.resize(refs, table, [5, 0, 9], 4)
    # row 1 gives page 2 back, row 2 takes the lowest free ids 1, 2, 4
    assert table == [[3, 0, -1], [-1, -1, -1], [1, 2, 4]]
    assert refs == [1, 1, 1, 1, 1] and not moves and not err
    assert pages.resize(refs, table, [5, 1, 9], 4)[1] == {"no_page"}
    assert table[1] == [-1, -1, -1]
    assert pages.resize(refs, table, [0, 0, 13], 4)[1] == {"length"}
    assert refs == [0, 1, 1, 0, 1]


def test_fork_by_hand():
    refs = [1, 1, 1, 0, 0, 0]
    table = [[2, 0, -1], [1, -1, -1], [-1] * 3]
    lens = [6, 4, 0]
    moves, err = pages.fork(refs, table, lens, [0, 0], [1, 2], 4)
    # page 1 of row 1 goes back first and is the first page given out
    assert table == [[2, 0, -1], [2, 1, -1], [2, 3, -1]]
    assert moves == [(0, 1), (0, 3)] and not err
    assert refs == [1, 1, 3, 1, 0, 0] and lens == [6, 6, 6]
    # a child named twice, a child that is a parent, a row outside the table, padding
    moves, err = pages.fork(refs, table, lens, [0, 0, 2, 0, -1], [1, 1, 0, 9, 2], 4)
    assert err == {"fork"} and moves == [(0, 1)]
    assert refs == _counts(refs, table)


def test_compact_by_hand():
    refs, table = [0, 2, 0, 1, 0, 1], [[5, 1], [1, 3], [-1, -1]]
    moves, err, used = pages.compact(refs, table)
    assert used == 3 and moves == [(3, 0), (5, 2)] and not err
    assert table == [[2, 1], [1, 0], [-1, -1]] and refs == [1, 2, 1, 0, 0, 0]
    assert pages.compact([0, 1], [[0, 1]])[1] == {"page"}


def test_counts_follow_the_table_through_random_calls():
    rng = random.Random(0)
    for _ in range(200):
        rows, width, n, ps = rng.randint(2, 6), rng.randint(1, 5), rng.randint(3, 30), 4
        refs, table, lens = [0] * n, [[-1] * width for _ in range(rows)], [0] * rows
        for _ in range(12):
            op = rng.choice(["resize", "fork", "compact"])
            if op == "resize":
                lens = [rng.randint(0, width * ps) for _ in range(rows)]
                _, err = pages.resize(refs, table, lens, ps)
                if err:      # a row that got too few pages ends where they do
                    for i, row in enumerate(table):
                        got = next((k for k, e in enumerate(row) if e < 0), width)
                        lens[i] = min(lens[i], got * ps)
                    pages.resize(refs, table, lens, ps)
            elif op == "fork":
                ids = rng.sample(range(rows), 2)
                pages.fork(refs, table, lens, [ids[0]], [ids[1]], ps)
            else:
                _, err, used = pages.compact(refs, table)
                assert not err and all(refs[:used]) and not any(refs[used:])
            assert refs == _counts(refs, table)
            for row, m in zip(table, lens):
                assert [e >= 0 for e in row] == [k < -(-m // ps) for k in range(width)]
