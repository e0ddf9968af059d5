"""The page operations on host arrays, one list entry after the other (oracle).

table int32 [n_slots][max_pages] (entries below 0 unused), refs int32
[n_pages]; both are changed in place.  Each function returns the error bits.
"""

from __future__ import annotations

import numpy as np

BAD_SEQUENCE, BAD_PAGE, NO_PAGES = 0x1, 0x4, 0x8


def _release(table, refs, slot):
    err = 0
    for c, e in enumerate(table[slot]):
        if e >= len(refs):
            err |= BAD_PAGE
        elif e >= 0:
            if refs[e] <= 0:
                err |= BAD_PAGE
            else:
                refs[e] -= 1
        table[slot, c] = -1
    return err


def free(table, refs, seqs):
    err = 0
    for s in seqs:
        err |= _release(table, refs, s) if 0 <= s < len(table) else BAD_SEQUENCE
    return err


def reserve(table, refs, seqs, lens, page_rows):
    err, wants, seen = 0, [], set()
    for s, n in zip(seqs, lens):
        if not 0 <= s < len(table) or s in seen or not 0 <= n <= table.shape[1] * page_rows:
            err |= BAD_SEQUENCE
        else:
            held = table[s, :-(-int(n) // page_rows)]
            err |= BAD_PAGE if (held >= len(refs)).any() else 0
            wants += [(s, c) for c in np.flatnonzero(held < 0)]
        seen.add(s)
    pages = np.flatnonzero(refs == 0)
    if len(wants) > len(pages):
        return err | NO_PAGES
    for (s, c), p in zip(wants, pages):
        table[s, c] = p
        refs[p] = 1
    return err


def fork(table, refs, parents, children, lens, page_rows):
    """(error bits, src, dst)"""
    err, seen, valid = 0, set(), []
    n_slots, max_pages = table.shape
    for p, c, n in zip(parents, children, lens):
        ok = (0 <= c < n_slots and 0 <= p < n_slots and c not in seen and c not in set(parents)
              and 0 <= n <= max_pages * page_rows)
        seen.add(c)
        e = 0 if ok else BAD_SEQUENCE
        if ok:
            held = table[p, :-(-int(n) // page_rows)]
            e = (BAD_SEQUENCE if (held < 0).any() else 0) | (BAD_PAGE if (held >= len(refs)).any() else 0)
        err |= e
        valid.append(e == 0)
    for c, ok in zip(children, valid):
        if ok:
            err |= _release(table, refs, c)
    pages = iter(np.flatnonzero(refs == 0))
    src = np.full(len(parents), -1, np.int32)
    dst = src.copy()
    for i, (p, c, n) in enumerate(zip(parents, children, lens)):
        if not valid[i]:
            continue
        full = int(n) // page_rows
        if n % page_rows:
            to = next(pages, None)
            if to is None:
                err |= NO_PAGES
                continue
            src[i], dst[i] = table[p, full], to
            table[c, full] = to
            refs[to] = 1
        table[c, :full] = table[p, :full]
        for e in table[p, :full]:
            refs[e] += 1
    return err, src, dst


def compact(table, refs):
    """(error bits, table after, refs after, src, dst, counts)"""
    n = len(refs)
    live = [p for p in range(n) if refs[p] > 0]
    n_live = len(live)
    movers = [p for p in live if p >= n_live]
    holes = [p for p in range(n_live) if refs[p] <= 0]
    to = dict(zip(movers, holes))
    err, out = 0, table.copy()
    for at, e in np.ndenumerate(table):
        if e >= n or e >= 0 and refs[e] <= 0:
            err |= BAD_PAGE
        elif e >= n_live:
            out[at] = to[e]
    refs_out = np.zeros_like(refs)
    for p in live:
        refs_out[to.get(p, p)] = refs[p]
    src = np.full(max(1, n // 2), -1, np.int32)
    dst = src.copy()
    src[:len(movers)], dst[:len(movers)] = movers, holes
    return err, out, refs_out, src, dst, np.array([n_live, len(movers)], np.int32)
