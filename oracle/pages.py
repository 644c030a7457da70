"""Page management of the paged cache by its definition, one page at a time.

``table`` is a list of rows of page ids (a row's valid entries), ``ref`` the rows that hold each
page, ``k`` / ``v`` the caches as [pages, tokens of a page, ...] arrays."""


def count(table, num_pages):
    ref = [0] * num_pages
    for row in table:
        for page in row:
            ref[page] += 1
    return ref


def copy(src, dst, caches):
    for s, d in zip(src, dst):
        if s >= 0 and d >= 0:
            for c in caches:
                c[d] = c[s]


def fork(table, ref, src, dst, cached, page_tokens, null_page, caches):
    free = [i for i, n in enumerate(ref) if n == 0 and i != null_page]
    for s, d in zip(src, dst):
        full, tail = divmod(int(cached[s]), page_tokens)
        row = list(table[s][:full])
        for page in row:
            ref[page] += 1
        if tail:
            page = free.pop(0)
            ref[page] = 1
            for c in caches:
                c[page][:tail] = c[table[s][full]][:tail]
            row.append(page)
        table[d] = row


def free(table, ref, rows):
    """Returns how many pages became free."""
    freed = 0
    for r in rows:
        for page in table[r]:
            ref[page] -= 1
            freed += ref[page] == 0
        table[r] = []
    return freed


def compact(table, ref, null_page, caches):
    """Returns (the new id of each page, the number of live pages)."""
    live = [i for i, n in enumerate(ref) if n > 0 and i != null_page]
    low = [i for i in range(len(ref)) if i != null_page][:len(live)]
    holes = [i for i in low if ref[i] <= 0]
    movers = [i for i in live if i not in set(low)]
    new = [i if ref[i] > 0 else -1 for i in range(len(ref))]
    new[null_page] = null_page
    for a, b in zip(movers, holes):
        new[a] = b
        ref[b], ref[a] = ref[a], 0
        for c in caches:
            c[b] = c[a]
    for row in table:
        row[:] = [new[p] for p in row]
    return new, len(live)
