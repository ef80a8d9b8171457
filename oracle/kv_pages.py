"""Oracle of the page operations of include/kv_pages.h: plain loops over rows and pages on
NumPy arrays, changed in place. Shares no code with the CUDA path.

`mutant` plants one mistake: 1: reserve gives pages out from the highest id; 2: a shared
page is not copied; 3: free keeps the page count of the kept tokens minus one; 4: compact
leaves the tables alone; 5: fork forgets the new owner."""
from __future__ import annotations

import numpy as np

ROW, LEN, PAGE, NO_PAGE, CHILD, REFS = 1, 2, 4, 8, 16, 32


def reserve(rows, old, new, table, page, refs, planes, mutant=0):
    status, plan = 0, []
    for r, a, b in zip(rows, old, new):
        need = []
        if r < 0 or r >= table.shape[0]:
            status |= ROW
        elif a < 0 or b < a or -(-b // page) > table.shape[1]:
            status |= LEN
        elif b > a:
            for c in range(a // page, -(-b // page)):
                e = int(table[r, c])
                if e >= len(refs):
                    status |= PAGE
                elif e < 0 or refs[e] > 1:
                    need.append(c)
        plan.append(need)
    free = [p for p in range(len(refs)) if refs[p] == 0]
    if mutant == 1:
        free = free[::-1]
    copies, at = [], 0
    stop = False
    changes = []
    for (r, a), need in zip(zip(rows, old), plan):
        if need and (stop or at + len(need) > len(free)):
            status |= NO_PAGE
            stop = True
            continue
        for c in need:
            changes.append((r, a, c, free[at]))
            at += 1
    for r, a, c, p in changes:
        e = int(table[r, c])
        if e >= 0:
            refs[e] -= 1
            if c * page < a and mutant != 2:
                copies.append((e, p))
        table[r, c] = p
        refs[p] = 1
    for s, d in copies:
        for x in planes:
            x[d] = x[s]
    return status


def fork(parents, children, lens, table, page, refs, mutant=0):
    status = 0
    n_tables, width = table.shape
    for a, b, n in zip(parents, children, lens):
        if not (0 <= a < n_tables and 0 <= b < n_tables):
            status |= ROW
        elif n < 0 or -(-n // page) > width:
            status |= LEN
        elif (table[b] >= 0).any():
            status |= CHILD
        else:
            for c in range(-(-n // page)):
                e = int(table[a, c])
                if e >= len(refs):
                    status |= PAGE
                    e = -1
                table[b, c] = e
                if e >= 0 and mutant != 5:
                    refs[e] += 1
    return status


def free(rows, keep, table, page, refs, mutant=0):
    status = 0
    for i, r in enumerate(rows):
        n = 0 if keep is None else int(keep[i])
        if not 0 <= r < table.shape[0]:
            status |= ROW
            continue
        if n < 0:
            status |= LEN
            continue
        for c in range(max(0, -(-n // page) - (mutant == 3)), table.shape[1]):
            e = int(table[r, c])
            if e < 0:
                continue
            table[r, c] = -1
            if e >= len(refs):
                status |= PAGE
            elif refs[e] <= 0:
                status |= REFS
            else:
                refs[e] -= 1
    return status


def compact(table, refs, planes, mutant=0):
    """Returns (status, new_ids, (live, moved))."""
    n = len(refs)
    live = sum(int(r > 0) for r in refs)
    movers = [p for p in range(live, n) if refs[p] > 0]
    holes = [p for p in range(live) if refs[p] <= 0]
    new = np.array([p if refs[p] > 0 else -1 for p in range(n)], np.int32)
    status = 0
    for a, b in zip(movers, holes):
        new[a] = b
        refs[b], refs[a] = refs[a], 0
        for x in planes:
            x[b] = x[a]
    if mutant != 4:
        for i in range(table.shape[0]):
            for c in range(table.shape[1]):
                e = int(table[i, c])
                if e >= n:
                    status |= PAGE
                elif e >= 0:
                    if new[e] < 0:
                        status |= REFS
                    else:
                        table[i, c] = new[e]
    return status, new, (live, len(movers))


def copy(src, dst, planes, n_pages):
    status = 0
    for s, d in zip(src, dst):
        if s < 0 and d < 0:
            continue
        if not (0 <= s < n_pages and 0 <= d < n_pages):
            status |= PAGE
            continue
        for x in planes:
            x[d] = x[s]
    return status


TOKENS = 64


def step(rows, old, new, table, page, num_pages, tokens, mutant=0):
    """(positions, token_table, slots, lens, starts, status) of a step's tokens, one after
    another. `mutant` 6: padding rows are row 0; 7: a token's length leaves itself out."""
    got = [[], [], [], []]
    starts, status = [0], 0
    for r, a, b in zip(rows, old, new):
        if not 0 <= r < table.shape[0]:
            status |= ROW
        elif a < 0 or b < a or b > table.shape[1] * page:
            status |= LEN
        else:
            for pos in range(a, b):
                if len(got[0]) == tokens:
                    status |= TOKENS
                    break
                e = int(table[r, pos // page])
                slot = -1
                if e < 0:
                    status |= NO_PAGE
                elif e >= num_pages:
                    status |= PAGE
                else:
                    slot = e * page + pos % page
                for x, y in zip(got, (pos, r, slot, pos + (mutant != 7))):
                    x.append(y)
        starts.append(len(got[0]))
    rest = tokens - len(got[0])
    for x, y in zip(got, (-1, 0 if mutant == 6 else -1, -1, 0)):
        x += [y] * rest
    return tuple(np.asarray(x, np.int32) for x in got) + (np.asarray(starts, np.int32), status)


def shared(rows, lens, starts, table, page, num_pages, mutant=0):
    """(prefix lengths, status). `mutant` 8: rows of length 0 count too."""
    out, status = [], 0
    for a, b in zip(starts, starts[1:]):
        if not 0 <= a <= b <= len(rows):
            status |= LEN
            out.append(0)
            continue
        live, bad = [], False
        for r, n in zip(rows[a:b], lens[a:b]):
            if n == 0 and mutant != 8:
                continue
            if not 0 <= r < table.shape[0]:
                status |= ROW
                bad = True
            elif n < 0 or n > table.shape[1] * page:
                status |= LEN
                bad = True
            else:
                live.append((r, n))
        pages = 0
        if len(live) > 1 and not bad:
            for c in range(min(n for _, n in live) // page):
                ids = {int(table[r, c]) for r, _ in live}
                if len(ids) > 1 or not 0 <= min(ids) < num_pages:
                    break
                pages += 1
        out.append(pages * page)
    return np.asarray(out, np.int32), status
