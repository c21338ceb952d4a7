"""The page operators one request after another, on Python lists."""
from __future__ import annotations

import random


def pages_of(tokens, page_tokens):
    return -(-tokens // page_tokens)


class Cache:
    def __init__(self, pages, rows, max_pages, page_tokens):
        self.refs = [0] * pages
        self.table = [[-1] * max_pages for _ in range(rows)]
        self.lengths = [0] * rows
        self.page_tokens = page_tokens

    def copy(self):
        c = Cache(0, 0, 0, self.page_tokens)
        c.refs, c.table, c.lengths = list(self.refs), [list(r) for r in self.table], list(self.lengths)
        return c

    def _row(self, row):
        return 0 <= row < len(self.table)

    def grow(self, rows, new_lengths):
        free = [p for p, n in enumerate(self.refs) if n <= 0]
        at, seen, granted = 0, set(), []
        for row, new in zip(rows, new_lengths):
            ok = self._row(row) and row not in seen and new >= self.lengths[row] and \
                pages_of(new, self.page_tokens) <= len(self.table[row])
            if self._row(row):
                seen.add(row)
            if ok:
                old = pages_of(self.lengths[row], self.page_tokens)
                need = pages_of(new, self.page_tokens) - old
                ok = need == 0 or at + need <= len(free)
                if ok:
                    for k in range(need):
                        self.table[row][old + k] = free[at + k]
                        self.refs[free[at + k]] = 1
                    self.lengths[row] = new
                at += need
            granted.append(int(ok))
        return granted

    def fork(self, parents, children):
        free = [p for p, n in enumerate(self.refs) if n <= 0]
        before, tables = list(self.lengths), [list(r) for r in self.table]
        at, seen, granted, src, dst = 0, set(), [], [], []
        for parent, child in zip(parents, children):
            ok = self._row(parent) and self._row(child) and child not in seen and before[child] == 0
            if self._row(child):
                seen.add(child)
            if ok:
                n = before[parent]
                whole, part = divmod(n, self.page_tokens)
                if part:
                    ok = at < len(free)
                    at += 1
            if ok:
                row = tables[parent][:whole]
                for p in row:
                    if 0 <= p < len(self.refs):
                        self.refs[p] += 1
                if part:
                    new = free[at - 1]
                    self.refs[new] = 1
                    src.append(tables[parent][whole])
                    dst.append(new)
                    row.append(new)
                self.table[child] = row + [-1] * (len(self.table[child]) - len(row))
                self.lengths[child] = n
            granted.append(int(ok))
        return granted, src, dst

    def free(self, rows):
        freed = 0
        for row in rows:
            if not self._row(row):
                continue
            n = pages_of(self.lengths[row], self.page_tokens)
            for i in range(min(n, len(self.table[row]))):
                p = self.table[row][i]
                if 0 <= p < len(self.refs):
                    freed += self.refs[p] == 1
                    self.refs[p] -= 1
                self.table[row][i] = -1
            self.lengths[row] = 0
        return freed

    def compact(self):
        used = [p for p, n in enumerate(self.refs) if n > 0]
        count = len(used)
        holes = [p for p in range(count) if self.refs[p] <= 0]
        behind = [p for p in used if p >= count]
        assert len(holes) == len(behind)
        remap = [p if n > 0 else -1 for p, n in enumerate(self.refs)]
        for a, b in zip(behind, holes):
            remap[a] = b
            self.refs[b], self.refs[a] = self.refs[a], 0
        for row in self.table:
            for i, p in enumerate(row):
                if 0 <= p < len(self.refs) and remap[p] >= 0:
                    row[i] = remap[p]
        return count, remap, behind, holes


def filled(seed, pages, rows, max_pages, page_tokens):
    """A cache after rows grew, forked and ended in no order."""
    rng = random.Random(seed)
    c = Cache(pages, rows, max_pages, page_tokens)
    for _ in range(4):
        some = rng.sample(range(rows), max(1, rows // 2))
        c.grow(some, [min(max_pages * page_tokens, c.lengths[r] + rng.randint(0, max(1, max_pages * page_tokens // 3)))
                      for r in some])
        empty = [r for r in range(rows) if not c.lengths[r]]
        c.fork([rng.randrange(rows) for _ in empty[::2]], empty[::2])
        c.free(rng.sample(range(rows), rows // 4))
    return c
