"""Oracle: page tables, reference counts and moves of pages (test infrastructure only).

Plain sequential models on Python lists.  ``refs[p]`` counts the table entries that
name page p.  Each function changes ``refs``, ``table`` and ``lens`` in place and returns
(moves, errors): the (source, destination) pairs of pages to copy and the set of
error names {"page", "length", "no_page", "fork"}.
"""


def _give_back(refs, page, errors):
    if refs[page] <= 0:
        errors.add("page")
    else:
        refs[page] -= 1


def _need(length, width, page_size, errors):
    n = -(-max(length, 0) // page_size)
    if n > width:
        errors.add("length")
    return min(n, width)


def resize(refs, table, lens, page_size):
    errors = set()
    need = [_need(n, len(row), page_size, errors) for n, row in zip(lens, table)]
    for row, n in zip(table, need):
        for k, e in enumerate(row):
            if e >= len(refs):
                errors.add("page")
                row[k] = -1
            elif e >= 0 and k >= n:
                _give_back(refs, e, errors)
                row[k] = -1
    free = [p for p, r in enumerate(refs) if r == 0]
    for row, n in zip(table, need):
        for k in range(n):
            if row[k] < 0:
                if free:
                    row[k] = free.pop(0)
                    refs[row[k]] = 1
                else:
                    errors.add("no_page")
    return [], errors


def fork(refs, table, lens, parents, children, page_size):
    errors, moves = set(), []
    n, width = len(table), len(table[0])
    named = [(p, c) for p, c in zip(parents, children) if p >= 0 and c >= 0]
    inside = [(p, c) for p, c in named if p < n and c < n]
    all_parents = {p for p, _ in inside}
    takes, seen = [], set()
    for p, c in named:
        ok = p < n and c < n and c not in seen and c not in all_parents
        if p < n and c < n:
            seen.add(c)
        if ok:
            takes.append((p, c))
        else:
            errors.add("fork")
    before = [list(r) for r in table]
    length = {}
    for p, c in takes:
        if lens[p] > width * page_size:
            errors.add("length")
        length[c] = min(max(lens[p], 0), width * page_size)
        for k in range(width):
            table[c][k] = -1
            if k < length[c] // page_size:
                e = before[p][k]
                if 0 <= e < len(refs):
                    refs[e] += 1
                    table[c][k] = e
                else:
                    errors.add("page")
    for p, c in takes:
        for e in before[c]:
            if e >= len(refs):
                errors.add("page")
            elif e >= 0:
                _give_back(refs, e, errors)
    free = [p for p, r in enumerate(refs) if r == 0]
    for p, c in takes:
        if length[c] % page_size:
            k = length[c] // page_size
            e = before[p][k]
            if not 0 <= e < len(refs):
                errors.add("page")
            elif free:
                table[c][k] = free.pop(0)
                refs[table[c][k]] = 1
                moves.append((e, table[c][k]))
            else:
                errors.add("no_page")
                length[c] = k * page_size
        lens[c] = length[c]
    return moves, errors


def compact(refs, table):
    """Also returns the number of used pages: (moves, errors, used)."""
    errors = set()
    used = sum(r > 0 for r in refs)
    holes = [p for p in range(used) if refs[p] <= 0]
    movers = [p for p in range(used, len(refs)) if refs[p] > 0]
    to = {p: p for p in range(used) if refs[p] > 0}
    to.update(zip(movers, holes))
    new = [0] * len(refs)
    for p, q in to.items():
        new[q] = refs[p]
    refs[:] = new
    for row in table:
        for k, e in enumerate(row):
            if e >= 0:
                row[k] = to.get(e, -1)
                if row[k] < 0:
                    errors.add("page")
    return list(zip(movers, holes)), errors, used
