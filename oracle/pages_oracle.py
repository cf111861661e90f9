"""Plain simulation of the cache's pages (numpy; test infrastructure). Every
function changes its arrays in place; the cache is a list of arrays [pages, Hkv,
page_size, ...]."""
from __future__ import annotations

import numpy as np


def _pages(n, page_size):
    return -(-n // page_size)


def compact(cache, table, starts, bases, keep, cu, dst_table=None):
    """Returns the new lengths."""
    page = cache[0].shape[2]
    to = table if dst_table is None else dst_table
    lens = np.zeros(len(cu) - 1, np.int64)
    for r in range(len(cu) - 1):
        rows = [[a[table[r, p // page], :, p % page].copy() for a in cache]
                for p in (starts[r] + keep[j] - bases[r] for j in range(cu[r], cu[r + 1]))]
        for k, row in enumerate(rows):
            at = starts[r] + k
            for a, x in zip(cache, row):
                a[to[r, at // page], :, at % page] = x
        lens[r] = starts[r] + len(rows)
    return lens


def shared_end(refs, table, lens, new_lens, page_size):
    """The rows that would grow from inside a page that others hold too."""
    return np.asarray([new_lens[r] > lens[r] and lens[r] % page_size != 0 and refs[table[r, lens[r] // page_size]] > 1
                       for r in range(len(lens))], bool)


def resize(refs, table, lens, new_lens, page_size):
    """False where pages ran out. Rows of shared_end() stay as they are."""
    held = shared_end(refs, table, lens, new_lens, page_size)
    free = iter(np.flatnonzero(refs == 0).tolist())
    left, ok = int((refs == 0).sum()), True
    refs0 = refs.copy()
    for r in range(len(lens)):
        if new_lens[r] < 0 or held[r]:
            continue
        have, need = _pages(lens[r], page_size), _pages(new_lens[r], page_size)
        if need > have:
            ok = ok and need - have <= left
            if not ok:
                continue
            left -= need - have
            for i in range(have, need):
                page = next(free)
                assert refs0[page] == 0
                table[r, i] = page
                refs[page] = 1
        for i in range(need, have):
            refs[table[r, i]] -= 1
        lens[r] = new_lens[r]
    return ok


def good_forks(lens, parents, children):
    """Which forks are taken: children above all before them, of length 0, from rows that are
    not themselves listed as children above all before them."""
    rows, top, listed = len(lens), -1, set()
    above = []
    for c in children:
        above.append(c > top)
        top = max(top, c)
        if above[-1]:
            listed.add(c)
    return [bool(a and 0 <= c < rows and 0 <= p < rows and p not in listed and lens[c] == 0) for p, c, a in zip(parents, children, above)]


def fork(cache, refs, table, lens, parents, children):
    """Children without a page stay as they are."""
    page = cache[0].shape[2]
    free = iter(np.flatnonzero(refs == 0).tolist())
    for p, c in zip(parents, children):
        n, whole = lens[p], lens[p] // page
        if n % page:
            fresh = next(free, None)
            if fresh is None:
                continue
            for a in cache:
                a[fresh, :, :n % page] = a[table[p, whole], :, :n % page]
            refs[fresh] = 1
        table[c, :whole] = table[p, :whole]
        if n % page:
            table[c, whole] = fresh
        for i in range(whole):
            refs[table[p, i]] += 1
        lens[c] = n
