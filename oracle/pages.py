"""The page operations of a paged cache, one row and one page at a time.

table: list of rows of page ids; refs: holders of each page (rows and other
owners); lens: positions of each row.  Row b holds its first ceil(lens[b] / 64)
entries.  Free pages (refs 0) are handed out from the lowest id up, in the
order of the rows.  Each function leaves its arguments alone and returns what
the operation leaves behind, with the pairs (from, to) of copied pages."""
TILE = 64


def held(n):
    return -(-n // TILE)


def _split_shared(pages, refs, rows):
    """rows: those that will write the partly filled page pages[b].  The ones that must take a copy: all but the
    first of a page's rows, and that one too where somebody else holds the page."""
    takers = []
    for b in rows:
        mine = [o for o in rows if pages[o] == pages[b]]
        if mine[0] != b or refs[pages[b]] > len(mine):
            takers.append(b)
    return takers


def fork(parent, table, refs, lens):
    """(table, refs, lens, pairs, short): short: rows that got no page for their copy."""
    refs, new_lens = list(refs), [lens[p] if p >= 0 else 0 for p in parent]
    rows = [list(r) for r in table]
    for b, p in enumerate(parent):
        if p >= 0:
            rows[b][:held(lens[p])] = table[p][:held(lens[p])]
    for b in range(len(parent)):
        for page in table[b][:held(lens[b])]:
            refs[page] -= 1
        for page in rows[b][:held(new_lens[b])]:
            refs[page] += 1
    part = [b for b in range(len(parent)) if new_lens[b] % TILE]
    last = {b: rows[b][new_lens[b] // TILE] for b in part}
    takers = _split_shared(last, refs, part)
    free = [p for p in range(len(refs)) if refs[p] == 0]
    pairs, short = [], []
    for k, b in enumerate(takers):
        refs[last[b]] -= 1
        t = new_lens[b] // TILE
        if k < len(free):
            rows[b][t] = free[k]
            refs[free[k]] = 1
            pairs.append((last[b], free[k]))
        else:
            rows[b][t] = -1
            new_lens[b] = t * TILE
            short.append(b)
    return rows, refs, new_lens, pairs, short


def resize(table, refs, lens, new_lens):
    """(table, refs, lens, pairs, short)."""
    rows, refs, got = [list(r) for r in table], list(refs), list(new_lens)
    for b, (n, m) in enumerate(zip(lens, new_lens)):
        for t in range(held(m), held(n)):
            refs[rows[b][t]] -= 1
            rows[b][t] = -1
    part = [b for b, (n, m) in enumerate(zip(lens, new_lens)) if m > n and n % TILE]
    last = {b: rows[b][lens[b] // TILE] for b in part}
    takers = _split_shared(last, refs, part)
    free = [p for p in range(len(refs)) if refs[p] == 0]
    pairs, short, at = [], [], 0
    for b, (n, m) in enumerate(zip(lens, new_lens)):
        want = (b in takers) + max(0, held(m) - held(n))
        mine, at = free[at:at + want], at + want
        if len(mine) < want:
            short.append(b)
        if b in takers:
            if not mine:
                got[b] = n
                continue
            page = mine.pop(0)
            refs[last[b]] -= 1
            refs[page] = 1
            rows[b][n // TILE] = page
            pairs.append((last[b], page))
        for t, page in enumerate(mine, held(n)):
            rows[b][t] = page
            refs[page] = 1
        if b in short:
            got[b] = (held(n) + len(mine)) * TILE
    return rows, refs, got, pairs, short


def compact(table, refs, lens):
    """(table, refs, map, n_live, pairs)."""
    live = [p for p, r in enumerate(refs) if r > 0]
    n = len(live)
    holes = [p for p in range(n) if refs[p] <= 0]
    pairs = list(zip([p for p in live if p >= n], holes))
    to = [p if r > 0 else -1 for p, r in enumerate(refs)]
    refs = list(refs)
    for src, dst in pairs:
        to[src] = dst
        refs[dst], refs[src] = refs[src], 0
    rows = [list(r) for r in table]
    for b, m in enumerate(lens):
        rows[b][:held(m)] = [to[p] for p in rows[b][:held(m)]]
    return rows, refs, to, n, pairs
