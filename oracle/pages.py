"""The pages of a paged cache, one step after another on the host.

Fork, reserve, free and compact as kvc.h describes them ("10.3 -- KV cache
implementation details", section 7: block tables, blocks shared by sequences
with a common prefix), in plain Python on lists: sequence after sequence, page
after page.  ``rows`` notes which rows a step copies, as (source block,
destination block, number of rows).
"""
from __future__ import annotations

PAGE = 16


class Pages:
    def __init__(self, table, refs):
        self.table = [[int(x) for x in row] for row in table]
        self.refs = [int(x) for x in refs]

    def fork(self, parent):
        old = [list(row) for row in self.table]
        for b, p in enumerate(parent):
            if not -1 <= p < len(old):
                continue
            row = [-1] * len(old[b]) if p < 0 else list(old[p])
            for x in row:
                if x >= 0:
                    self.refs[x] += 1
            for x in old[b]:
                if x >= 0:
                    self.refs[x] -= 1
            self.table[b] = row

    def reserve(self, length, grown):
        """The rows copied, or None where the free blocks do not suffice."""
        limit = PAGE * len(self.table[0])
        refs, todo = list(self.refs), []
        for b, (n, m) in enumerate(zip(length, grown)):
            if not 0 <= n < m <= limit:
                continue
            if n % PAGE and self.table[b][n // PAGE] < 0:
                continue
            for j in range(n // PAGE, -(-m // PAGE)):
                x = self.table[b][j]
                if x < 0:
                    todo.append((b, j, None, 0))
                elif refs[x] > 1:   # shared: b leaves it
                    refs[x] -= 1
                    todo.append((b, j, x, n % PAGE if j == n // PAGE else 0))
        free = [x for x, r in enumerate(self.refs) if r == 0]
        if len(todo) > len(free):
            return None
        copied = []
        for (b, j, old, rows), page in zip(todo, free):
            self.table[b][j] = page
            refs[page] = 1
            if rows:
                copied.append((old, page, rows))
        self.refs = refs
        return copied

    def free(self, keep):
        limit = PAGE * len(self.table[0])
        for b, n in enumerate(keep):
            if not 0 <= n <= limit:
                continue
            for j in range(-(-n // PAGE), len(self.table[b])):
                if self.table[b][j] >= 0:
                    self.refs[self.table[b][j]] -= 1
                self.table[b][j] = -1

    def compact(self):
        """(pairs of blocks moved, live pages)."""
        live = sum(r > 0 for r in self.refs)
        holes = [x for x in range(live) if self.refs[x] <= 0]
        movers = [x for x in range(live, len(self.refs)) if self.refs[x] > 0]
        to = dict(zip(movers, holes))
        for a, b in to.items():
            self.refs[b], self.refs[a] = self.refs[a], 0
        self.table = [[to.get(x, x) for x in row] for row in self.table]
        return list(to.items()), live

    def check(self):
        """Every count is the number of entries that name the block."""
        count = [0] * len(self.refs)
        for row in self.table:
            for x in row:
                if x >= 0:
                    count[x] += 1
        return count == self.refs
