"""Page bookkeeping of a paged cache, one step at a time in plain Python: what
the fd_pages_* calls leave behind.  ``Books`` holds a block table (rows of page
numbers, -1 for none), lengths and reference counts."""
from __future__ import annotations

import numpy as np


class Books:
    def __init__(self, table, lengths, refs, page_size):
        self.table = np.array(table, dtype=np.int32)
        self.lengths = np.array(lengths, dtype=np.int32)
        self.refs = np.array(refs, dtype=np.int32)
        self.ps = int(page_size)
        self.cap = self.table.shape[1] * self.ps

    def _pages(self, positions):
        return -(-int(positions) // self.ps)

    def _len(self, b):
        return min(max(int(self.lengths[b]), 0), self.cap)

    def _release(self, b, first):
        for j in range(first, self.table.shape[1]):
            if 0 <= self.table[b, j] < len(self.refs):
                self.refs[self.table[b, j]] -= 1
            self.table[b, j] = -1

    def consistent(self):
        """refs is what the table says."""
        named = self.table[self.table >= 0]
        return (np.bincount(named, minlength=len(self.refs)) == self.refs).all()

    def free(self, seqs=None, lengths=None):
        seqs = range(len(self.table)) if seqs is None else seqs
        for i, b in enumerate(seqs):
            if not 0 <= b < len(self.table):
                continue
            L = 0 if lengths is None else min(self._len(b), max(int(lengths[i]), 0))
            self._release(b, self._pages(L))
            self.lengths[b] = L

    def fork(self, src, dst, lengths=None):
        n, B = len(src), len(self.table)
        rows, lens = self.table.copy(), [self._len(b) for b in range(B)]
        for i in range(n):
            s, d = int(src[i]), int(dst[i])
            if not (0 <= s < B and 0 <= d < B) or s == d or d in dst[:i]:
                continue
            if any(src[o] == d and dst[o] != d for o in range(n) if o != i):
                continue
            L = lens[s] if lengths is None else min(lens[s], max(int(lengths[i]), 0))
            for j in range(self._pages(L)):
                if 0 <= rows[s, j] < len(self.refs):
                    self.refs[rows[s, j]] += 1
            self._release(d, 0)
            self.table[d, :self._pages(L)] = rows[s, :self._pages(L)]
            self.lengths[d] = L

    def reorder(self, src):
        B = len(self.table)
        rows, lens, P = self.table.copy(), [self._len(b) for b in range(B)], len(self.refs)
        taken = []
        for b in range(B):
            s = int(src[b])
            if s == b or s >= B:
                taken.append((list(rows[b]), int(self.lengths[b])))
                continue
            L = lens[s] if s >= 0 else 0
            held = [int(e) if 0 <= e < P else -1 for e in rows[max(s, 0), :self._pages(L)]]
            taken.append((held + [-1] * (rows.shape[1] - len(held)), L))
        for b, (row, L) in enumerate(taken):
            for old, new in zip(rows[b], row):
                if old != new:
                    if 0 <= old < P:
                        self.refs[old] -= 1
                    if 0 <= new < P:
                        self.refs[new] += 1
            self.table[b] = row
            self.lengths[b] = L

    def reserve(self, n_new):
        """Returns the pairs (old, new) to copy, or minus the missing pages."""
        B = len(self.table)
        n_new = [n_new] * B if np.isscalar(n_new) else n_new
        spans = []
        for b in range(B):
            L = self._len(b)
            end = min(L + max(int(n_new[b]), 0), self.cap)
            spans += [(b, j) for j in range(L // self.ps, self._pages(end) if end > L else 0)]
        P = len(self.refs)
        writers = {}
        for b, j in spans:
            e = int(self.table[b, j])
            if 0 <= e < P and self.refs[e] > 1:
                writers.setdefault(e, []).append((b, j))
        moves = []
        for b, j in spans:
            e = int(self.table[b, j])
            if not 0 <= e < P:
                moves.append((b, j, -1))
            elif e in writers and not (len(writers[e]) == self.refs[e] and writers[e][0] == (b, j)):
                moves.append((b, j, e))
        spare = [p for p in range(P) if self.refs[p] <= 0]
        if len(moves) > len(spare):
            return -(len(moves) - len(spare))
        pairs = []
        for (b, j, old), new in zip(moves, spare):
            if old >= 0:
                self.refs[old] -= 1
                if j * self.ps < self._len(b):
                    pairs.append((old, new))
            self.refs[new] = 1
            self.table[b, j] = new
        return pairs

    def compact(self):
        used = [p for p in range(len(self.refs)) if self.refs[p] > 0]
        n = len(used)
        holes = [p for p in range(n) if self.refs[p] <= 0]
        pairs = list(zip([p for p in used if p >= n], holes))
        goes = np.arange(len(self.refs) + 1)       # the last: for entries of -1
        goes[-1] = -1
        for a, b in pairs:
            self.refs[b], self.refs[a] = self.refs[a], 0
            goes[a] = b
        self.table = goes[self.table].astype(np.int32)
        return pairs
