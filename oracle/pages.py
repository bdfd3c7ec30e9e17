"""Plain Python model of the page pool (pkv_pages_*): lists and loops, from the definitions.

A pool is (table, lens, refs, page_size); every call returns the new pool and its outputs,
or raises Refused with the code the library records, the pool unchanged (free goes entry by
entry and never refuses)."""
from __future__ import annotations

import numpy as np

OOM, BOUNDS = 4, 5


class Refused(Exception):
    def __init__(self, code):
        super().__init__(code)
        self.code = code


class Pool:
    def __init__(self, table, lens, refs, page_size):
        self.table, self.lens, self.refs, self.P = (np.array(x, dtype=np.int64) for x in (table, lens, refs, page_size))
        self.P = int(page_size)

    def copy(self):
        return Pool(self.table.copy(), self.lens.copy(), self.refs.copy(), self.P)

    def pages(self, row):
        return -(-int(self.lens[row]) // self.P)

    def _row(self, row):
        if not 0 <= row < len(self.lens) or not 0 <= self.lens[row] or self.pages(row) > self.table.shape[1]:
            raise Refused(BOUNDS)

    def _take(self, need):
        ids = [i for i in range(len(self.refs)) if self.refs[i] == 0][:need]
        if len(ids) < need:
            raise Refused(OOM)
        return ids

    def extend(self, rows, add, capacity=None):
        rows, add = [int(r) for r in rows], [int(a) for a in add]
        for r, a in zip(rows, add):
            self._row(r)
            if a < 0 or -(-(int(self.lens[r]) + a) // self.P) > self.table.shape[1]:
                raise Refused(BOUNDS)
        if len(set(rows)) < len(rows) or (capacity is not None and sum(add) > capacity):
            raise Refused(BOUNDS)
        need = [-(-(int(self.lens[r]) + a) // self.P) - self.pages(r) for r, a in zip(rows, add)]
        ids, new, slots = iter(self._take(sum(need))), self.copy(), []
        for r, a, k in zip(rows, add, need):
            for c in range(self.pages(r), self.pages(r) + k):
                new.table[r, c] = next(ids)
                new.refs[new.table[r, c]] = 1
            new.lens[r] += a
            slots += [int(new.table[r, t // self.P]) * self.P + t % self.P for t in range(int(self.lens[r]), int(new.lens[r]))]
        return new, slots

    def fork(self, parents, children):
        parents, children = [int(p) for p in parents], [int(c) for c in children]
        for p, c in zip(parents, children):
            self._row(c)
            self._row(p)
            if self.lens[c] != 0:
                raise Refused(BOUNDS)
        if len(set(children)) < len(children):
            raise Refused(BOUNDS)
        ids = iter(self._take(sum(int(self.lens[p]) % self.P > 0 for p in parents)))
        new, src, dst = self.copy(), [], []
        for p, c in zip(parents, children):
            full, part = divmod(int(self.lens[p]), self.P)
            new.table[c, :full] = self.table[p, :full]
            for page in self.table[p, :full]:
                new.refs[page] += 1
            src.append(int(self.table[p, full]) if part else -1)
            dst.append(next(ids) if part else -1)
            if part:
                new.table[c, full] = dst[-1]
                new.refs[dst[-1]] = 1
            new.lens[c] = self.lens[p]
        return new, src, dst

    def free(self, rows):
        """Entry by entry: self.bad counts the rows that are skipped and the ids and counts
        that are not what they should be."""
        new = self.copy()
        new.bad = 0
        for r in (int(r) for r in rows):
            try:
                new._row(r)
            except Refused:
                new.bad += 1
                continue
            for page in self.table[r, : new.pages(r)]:
                if 0 <= page < len(self.refs) and new.refs[page] > 0:
                    new.refs[page] -= 1
                else:
                    new.bad += 1
            new.lens[r] = 0
        return new

    def compact(self, max_moves=None):
        n = int((self.refs != 0).sum())
        src = [i for i in range(n, len(self.refs)) if self.refs[i] != 0]
        dst = [i for i in range(n) if self.refs[i] == 0]
        if max_moves is not None and len(src) > max_moves:
            raise Refused(BOUNDS)
        to, new = dict(zip(src, dst)), self.copy()
        for a, z in to.items():
            new.refs[z], new.refs[a] = self.refs[a], 0
        for r in range(len(self.lens)):
            for c in range(self.pages(r)):
                new.table[r, c] = to.get(int(self.table[r, c]), self.table[r, c])
        return new, src, dst
