"""A paged cache's bookkeeping with plain Python lists: one set of rules, no vector code."""
from __future__ import annotations

import numpy as np


class Cache:
    """k, v: [layers, pages, page_size, heads, dim] numpy arrays of any dtype, changed in place."""

    def __init__(self, k, v, refs, table):
        self.k, self.v, self.refs, self.table = k, v, refs, table
        self.ps = k.shape[2]

    def _free(self):
        return [g for g in range(len(self.refs)) if self.refs[g] == 0]

    def _pages(self, n):
        return -(-n // self.ps)

    def reserve(self, lens, extra):
        ok, asked, free = [], 0, self._free()
        for i, (n, more) in enumerate(zip(lens, extra)):
            if n < 0 or more < 0 or self._pages(n + more) > self.table.shape[1]:
                ok.append(0)
                continue
            lack = [e for e in range(self._pages(n + more)) if self.table[i, e] < 0]
            asked += len(lack)
            ok.append(int(asked <= len(free) or not lack))
            if ok[-1]:
                for e, g in zip(lack, free[asked - len(lack):asked]):
                    self.table[i, e] = g
                    self.refs[g] = 1
        return np.asarray(ok)

    def _at(self, i, slot):
        return self.table[i, slot // self.ps], slot % self.ps

    def append(self, k_new, v_new, lens, offsets, layer=0):
        for i in range(len(lens)):
            for c in range(offsets[i + 1] - offsets[i]):
                g, s = self._at(i, lens[i] + c)
                if g >= 0:
                    self.k[layer:layer + len(k_new), g, s] = k_new[:, offsets[i] + c]
                    self.v[layer:layer + len(v_new), g, s] = v_new[:, offsets[i] + c]

    def _drop(self, i, first):
        for e in range(first, self.table.shape[1]):
            if self.table[i, e] >= 0:
                self.refs[self.table[i, e]] -= 1
                self.table[i, e] = -1

    def commit(self, lens, path, accept_len):
        new = []
        for i, a in enumerate(accept_len):
            for j in range(max(a, 0)):
                (g, s), (h, t) = self._at(i, lens[i] + path[i, j]), self._at(i, lens[i] + 1 + j)
                self.k[:, h, t] = self.k[:, g, s]
                self.v[:, h, t] = self.v[:, g, s]
            new.append(lens[i] + 1 + a if a >= 0 else lens[i])
            self._drop(i, self._pages(new[-1]))
        return np.asarray(new)

    def fork(self, lens, src, dst):
        ok, free, asked = [], self._free(), 0
        before = lens.copy()
        for a, b in zip(src, dst):
            n = before[a]
            full, part = n // self.ps, n % self.ps
            if part:
                asked += 1
                if asked > len(free):
                    ok.append(0)
                    continue
                g = free[asked - 1]
                self.table[b, full], self.refs[g] = g, 1
                self.k[:, g, :part] = self.k[:, self.table[a, full], :part]
                self.v[:, g, :part] = self.v[:, self.table[a, full], :part]
            for e in range(full):
                self.table[b, e] = self.table[a, e]
                self.refs[self.table[a, e]] += 1
            lens[b] = n
            ok.append(1)
        return np.asarray(ok)

    def reorder(self, lens, src):
        """Rows become copies of rows src; 1 if that could be done."""
        R, old, before = len(src), self.table.copy(), lens.copy()
        refs = self.refs.copy()
        for j in range(R):
            if j not in list(src):
                for e in range(self.table.shape[1]):
                    if old[j, e] >= 0:
                        refs[old[j, e]] -= 1
        free, copies = [g for g in range(len(refs)) if refs[g] == 0], []
        rows = np.full_like(old, -1)
        for j, s in enumerate(src):
            if s < 0:
                continue
            keeper = s if src[s] == s else list(src).index(s)
            if j == keeper:
                rows[j] = old[s]
                continue
            full, part = before[s] // self.ps, before[s] % self.ps
            rows[j, :full] = old[s, :full]
            for e in range(full):
                refs[old[s, e]] += 1
            if part:
                if not free:
                    return 0
                rows[j, full] = free.pop(0)
                refs[rows[j, full]] = 1
                copies.append((rows[j, full], old[s, full], part))
        for to, of, part in copies:
            self.k[:, to, :part] = self.k[:, of, :part]
            self.v[:, to, :part] = self.v[:, of, :part]
        self.table[:], self.refs[:] = rows, refs
        lens[:] = [before[s] if s >= 0 else 0 for s in src]
        return 1

    def release(self, lens, seqs):
        for i in seqs:
            self._drop(i, 0)
            lens[i] = 0
