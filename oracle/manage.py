"""Page management of the cache, one page and one entry at a time.

State: `ref` (references per page), `table` (rows of page ids, -1 = none),
`lens`, and `data`, a list with whatever stands for each page's contents.  Every
function changes the state in place and returns the set of errors it met
("bounds", "pages").
"""


class State:
    def __init__(self, num_phys, rows, max_pages, ps):
        self.ps = ps
        self.ref = [0] * num_phys
        self.table = [[-1] * max_pages for _ in range(rows)]
        self.lens = [0] * rows
        self.data = [None] * num_phys

    def free_ids(self):
        return [p for p, r in enumerate(self.ref) if r == 0]


def _release(s, row, p, errors):
    e, s.table[row][p] = s.table[row][p], -1
    if e < 0:
        return
    if e >= len(s.ref) or s.ref[e] <= 0:
        errors.add("bounds")
    else:
        s.ref[e] -= 1


def copy(s, src, dst):
    errors, todo = set(), []
    n = len(s.data)
    fine = [0 <= a < n and 0 <= b < n for a, b in zip(src, dst)]
    for i, (a, b) in enumerate(zip(src, dst)):
        if not fine[i]:
            errors.add("bounds")
        elif a != b:
            others = [j for j in range(len(src)) if j != i and fine[j] and src[j] != dst[j]]
            if any(dst[j] == b or src[j] == b for j in others):
                errors.add("bounds")
            else:
                todo.append((b, s.data[a]))
    for b, x in todo:
        s.data[b] = x
    return errors


def fork(s, src, dst):
    errors = set()
    rows, ps = len(s.table), s.ps
    fine = [0 <= a < rows and 0 <= b < rows and dst.count(b) == 1 and b not in src for a, b in zip(src, dst)]
    if not all(fine):
        errors.add("bounds")
    for i, b in enumerate(dst):
        if fine[i]:
            for p in range(len(s.table[b])):
                _release(s, b, p, errors)
    free = iter(s.free_ids())
    plan = []
    for i, (a, b) in enumerate(zip(src, dst)):
        if not fine[i]:
            continue
        L, fresh = s.lens[a], None
        if not 0 <= L <= len(s.table[a]) * ps:
            errors.add("bounds")
            plan.append((a, b, None, 0))
            continue
        last = s.table[a][L // ps] if L % ps else -1
        if last >= len(s.ref):
            errors.add("bounds")
        elif last >= 0:
            fresh = next(free, -1)
        if fresh == -1:
            errors.add("pages")
            plan.append((a, b, None, 0))
        else:
            plan.append((a, b, fresh, L))
    for a, b, fresh, L in plan:
        row = [-1] * len(s.table[b])
        for p in range(L // ps):
            e = s.table[a][p]
            if e >= len(s.ref):
                errors.add("bounds")
            elif e >= 0:
                row[p] = e
                s.ref[e] += 1
        if fresh is not None:
            row[L // ps] = fresh
            s.ref[fresh] = 1
            s.data[fresh] = s.data[s.table[a][L // ps]]
        s.table[b], s.lens[b] = row, L
    return errors


def free(s, rows, window=None, sinks=0):
    errors = set()
    for b in range(len(s.table)) if rows is None else rows:
        if not 0 <= b < len(s.table):
            errors.add("bounds")
            continue
        for p in range(len(s.table[b])):
            tokens = range(p * s.ps, (p + 1) * s.ps)
            if window is None or not any(t < sinks or t >= s.lens[b] - window for t in tokens):
                _release(s, b, p, errors)
        if window is None:
            s.lens[b] = 0
    return errors


def reserve(s, lens):
    errors = set()
    free = s.free_ids()
    spent = False
    for b, want in enumerate(lens):
        first, last = -(-s.lens[b] // s.ps), -(-max(want, 0) // s.ps)
        if last > len(s.table[b]):
            errors.add("bounds")
            continue
        need = [p for p in range(first, last) if s.table[b][p] < 0]
        if need and (spent or len(need) > len(free)):
            spent = True
            errors.add("pages")
            continue
        for p in need:
            s.table[b][p] = free.pop(0)
            s.ref[s.table[b][p]] = 1
    return errors


def compact(s):
    errors = set()
    live = sum(r != 0 for r in s.ref)
    used = [r != 0 for r in s.ref]
    holes = [p for p in range(live) if s.ref[p] == 0]
    movers = [p for p in range(live, len(s.ref)) if s.ref[p] != 0]
    to = dict(zip(movers, holes))
    for a, b in to.items():
        s.data[b] = s.data[a]
        s.ref[b], s.ref[a] = s.ref[a], 0
    for row in s.table:
        for p, e in enumerate(row):
            if e >= len(used) or e >= 0 and not used[e]:
                errors.add("bounds")
            elif e in to:
                row[p] = to[e]
    return live, errors
