"""The page operators of a cache as the header describes them, one entry after the other, on numpy arrays."""
import numpy as np

ERR = {"SEQ": 1 << 8, "CHILD": 1 << 9, "PAGE": 1 << 10, "NO_PAGES": 1 << 11}


class Book:
    def __init__(self, table, refcounts, lengths=None, pools=()):
        self.table, self.refs = np.array(table, dtype=np.int64), np.array(refcounts, dtype=np.int64)
        self.lengths = None if lengths is None else np.array(lengths, dtype=np.int64)
        self.pools = [np.array(p) for p in pools]
        self.status = 0

    @property
    def shape(self):
        return (*self.table.shape, len(self.refs))

    def _free(self):
        return [int(p) for p in np.flatnonzero(self.refs <= 0)]

    def reserve(self, seqs, counts):
        S, M, P = self.shape
        todo, rows, seen = [], np.full((len(seqs), M), -1), set()
        for k, (s, c) in enumerate(zip(seqs, counts)):
            if not 0 <= s < S or s in seen:
                self.status |= ERR["SEQ"]
            elif not 0 <= c <= M:
                self.status |= ERR["PAGE"]
            else:
                todo.append((k, s, [j for j in range(c) if self.table[s, j] < 0]))
            seen.add(s)
        free, asked = self._free(), 0
        n_free = len(free)
        for k, s, need in todo:
            asked += len(need)
            if asked <= n_free:
                for j in need:
                    page = free.pop(0)
                    self.table[s, j], self.refs[page] = page, 1
            else:
                self.status |= ERR["NO_PAGES"]
            rows[k] = self.table[s]
        return rows

    def fork(self, parents, children, page_tokens):
        S, M, P = self.shape
        table, lengths = self.table.copy(), None if self.lengths is None else self.lengths.copy()
        rows, seen, free, asked = np.full((len(children), M), -1), set(), self._free(), 0
        n_free, copies = len(free), []
        for k, (p, c) in enumerate(zip(parents, children)):
            again, _ = c in seen, seen.add(c)
            if not 0 <= p < S or not 0 <= c < S or p == c or again:
                self.status |= ERR["SEQ"]
                continue
            if (table[c] >= 0).any():
                self.status |= ERR["CHILD"]
                continue
            n = M if page_tokens == 0 else -(-int(lengths[p]) // page_tokens)
            if (page_tokens and (lengths[p] < 0 or n > M or (table[p, :n] < 0).any())) or (table[p, :n] >= P).any():
                self.status |= ERR["PAGE"]
                continue
            own = [j for j in range(n) if table[p, j] >= 0 and (page_tokens == 0 or (j == n - 1 and lengths[p] % page_tokens))]
            asked += len(own)
            if asked > n_free:
                self.status |= ERR["NO_PAGES"]
                if lengths is not None:
                    self.lengths[c] = 0
                continue
            for j in range(n):
                if j in own:
                    page = free.pop(0)
                    copies.append((int(table[p, j]), page))
                    self.refs[page], rows[k, j] = 1, page
                elif table[p, j] >= 0:
                    self.refs[table[p, j]] += 1
                    rows[k, j] = table[p, j]
            self.table[c] = rows[k]
            if lengths is not None:
                self.lengths[c] = lengths[p]
        self._move(copies)
        return rows

    def _move(self, copies):
        for pool in self.pools:
            data = [pool[s].copy() for s, _ in copies]
            for (_, d), v in zip(copies, data):
                pool[d] = v

    def free(self, seqs):
        S, M, P = self.shape
        for s in seqs:
            if not 0 <= s < S:
                self.status |= ERR["SEQ"]
                continue
            for j in range(M):
                e, self.table[s, j] = int(self.table[s, j]), -1
                if e >= P or (e >= 0 and self.refs[e] <= 0):
                    self.status |= ERR["PAGE"]
                elif e >= 0:
                    self.refs[e] -= 1
            if self.lengths is not None:
                self.lengths[s] = 0

    def compact(self):
        S, M, P = self.shape
        live = self.refs > 0
        L = int(live.sum())
        movers, holes = [p for p in range(L, P) if live[p]], [p for p in range(L) if not live[p]]
        remap = np.where(live, np.arange(P), -1)
        refs = self.refs.copy()
        for s, d in zip(movers, holes):
            remap[s], refs[d] = d, self.refs[s]
        refs[L:] = 0
        if ((self.table < -1) | (self.table >= P)).any():
            self.status |= ERR["PAGE"]
        ok = (self.table >= 0) & (self.table < P)
        self.table = np.where(ok, remap[np.where(ok, self.table, 0)] if P else -1, -1)
        self.refs = refs
        self._move(list(zip(movers, holes)))
        return remap, L
