"""The pages of a paged cache, entry by entry in plain Python: rows of a block
table forked and dropped, pages taken for new tokens, the pages in use moved to
the front of the pool.  A table is a list of rows, each a list of the pages that
it holds; refs a list of counts."""
from __future__ import annotations


def pages_of(length, page):
    return -(-length // page)


def fork(table, lens, parents, refs):
    """New (table, lens, refs)."""
    refs = list(refs)
    new = [(list(table[p]), lens[p]) if p >= 0 else ([], 0) for p in parents]
    for row, _ in new:
        for p in row:
            refs[p] += 1
    for row in table:
        for p in row:
            refs[p] -= 1
    return [r for r, _ in new], [n for _, n in new], refs


def extend(table, lens, refs, n_new, page):
    """New (table, lens, refs), copies, pages taken, positions and slots of the new tokens; None with too few free pages."""
    table, lens, refs = [list(r) for r in table], list(lens), list(refs)
    free = [p for p, r in enumerate(refs) if r == 0]
    holders = {}                     # partly filled last page -> rows that go on in it
    for r, n in enumerate(n_new):
        if n > 0 and lens[r] % page:
            holders.setdefault(table[r][-1], []).append(r)
    keeps = {rows[0] for p, rows in holders.items() if refs[p] == len(rows)}
    taken, copies, at, slots = 0, [], [], []
    drops = []
    for r, n in enumerate(n_new):
        if n > 0 and lens[r] % page and refs[table[r][-1]] > 1 and r not in keeps:
            if taken == len(free):
                return None
            old, new = table[r][-1], free[taken]
            taken += 1
            copies.append((old, new))
            drops.append(old)
            refs[new] += 1
            table[r][-1] = new
        for pos in range(lens[r], lens[r] + n):
            if pos % page == 0:
                if taken == len(free):
                    return None
                table[r].append(free[taken])
                refs[free[taken]] += 1
                taken += 1
            at.append(pos)
            slots.append(table[r][pos // page] * page + pos % page)
        lens[r] += n
    for p in drops:
        refs[p] -= 1
    return table, lens, refs, copies, taken, at, slots


def compact(table, refs):
    """New (table, refs), copies, pages in use."""
    live = [p for p, r in enumerate(refs) if r > 0]
    L = len(live)
    moves = list(zip([p for p in live if p >= L], [p for p in range(L) if refs[p] == 0]))
    to = dict(moves)
    out = list(refs)
    for a, b in moves:
        out[b], out[a] = refs[a], 0
    return [[to.get(p, p) for p in row] for row in table], out, moves, L
