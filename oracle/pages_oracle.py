"""Plain Python oracle of the page tables: one request, one entry, one page
after the other.  Written from the definitions alone.  Test infrastructure only.

State: refs [n_pages], table [n_req][width], lens [n_req], lists of ints that
the functions change in place."""
from __future__ import annotations


def entries(length, page, width):
    """Entries that a request holds, None for a length out of range."""
    if length < 0 or length > min(width * page, 2 ** 31 - 1):
        return None
    return -(-length // page)


def _add(refs, page, by):
    if 0 <= page < len(refs):
        refs[page] += by


def resize(refs, table, lens, want, page):
    """Returns (copies, missing)."""
    n, width = len(lens), len(table[0]) if table else 1
    has = [entries(x, page, width) for x in lens]
    needs = [entries(x, page, width) for x in want]
    sound = [h is not None and w is not None for h, w in zip(has, needs)]
    for r in range(n):
        if sound[r] and want[r] < lens[r]:
            for j in range(needs[r], has[r]):
                _add(refs, table[r][j], -1)
                table[r][j] = -1
            lens[r] = want[r]
    grow = [r for r in range(n) if sound[r] and want[r] > lens[r]]
    part = {r: table[r][has[r] - 1] for r in grow if lens[r] % page and 0 <= table[r][has[r] - 1] < len(refs)}
    plan = []
    for r in grow:
        copy = False
        if r in part and refs[part[r]] > 1:
            all_of_them = [x for x in part if part[x] == part[r]]
            copy = not (len(all_of_them) == refs[part[r]] and all_of_them[0] == r)
        plan.append((r, copy))
    free = [p for p, c in enumerate(refs) if c == 0]
    total = sum(needs[r] - has[r] + c for r, c in plan)
    if total > len(free):
        return [], total - len(free)
    copies = []
    for r, copy in plan:
        if copy:
            new = free.pop(0)
            copies.append((part[r], new))
            refs[part[r]] -= 1
            refs[new] = 1
            table[r][has[r] - 1] = new
        for j in range(has[r], needs[r]):
            new = free.pop(0)
            refs[new] = 1
            table[r][j] = new
        lens[r] = want[r]
    return copies, 0


def fork(refs, table, lens, parents, page):
    n, width = len(lens), len(table[0])
    old_table, old_lens = [list(row) for row in table], list(lens)
    for r in range(n):
        p = parents[r]
        if p == r or p >= n or (p >= 0 and entries(old_lens[p], page, width) is None):
            continue
        has = entries(old_lens[r], page, width) or 0
        for j in range(has):
            _add(refs, old_table[r][j], -1)
            table[r][j] = -1
        lens[r] = 0
        if p >= 0:
            for j in range(entries(old_lens[p], page, width)):
                _add(refs, old_table[p][j], 1)
                table[r][j] = old_table[p][j]
            lens[r] = old_lens[p]


def compact(refs, table, lens, page, most):
    """Returns (copies, held, page_map)."""
    held = sum(c > 0 for c in refs)
    page_map = [-1 if c == 0 else p for p, c in enumerate(refs)]
    copies = []
    while len(copies) < most:
        top = max((p for p, c in enumerate(refs) if c > 0), default=-1)
        low = min((p for p, c in enumerate(refs) if c == 0), default=len(refs))
        if top <= low:
            break
        copies.append((top, low))
        refs[low], refs[top] = refs[top], 0
        page_map[top] = low
    for r in range(len(lens)):
        for j in range(entries(lens[r], page, len(table[r])) or 0):
            if 0 <= table[r][j] < len(refs) and page_map[table[r][j]] >= 0:
                table[r][j] = page_map[table[r][j]]
    return copies, held, page_map
