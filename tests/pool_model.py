"""A page pool in plain Python and numpy: what the pa_pool calls are to do, page by page."""
import numpy as np


class PoolModel:
    """tables [rows, width], ctx [rows], refs [blocks]; pages: arrays [layers, blocks, bs, ...] and
    scales: arrays [layers, blocks, heads, bs]."""

    def __init__(self, rows, width, blocks, bs, pages=(), scales=()):
        self.tables = np.full((rows, width), -1, np.int32)
        self.ctx = np.zeros(rows, np.int32)
        self.refs = np.zeros(blocks, np.int32)
        self.bs, self.pages, self.scales = bs, list(pages), list(scales)

    def check(self):
        """Counts are the entries that name a page; entries end where the context ends."""
        want = np.zeros_like(self.refs)
        for row, n in zip(self.tables, self.ctx):
            k = -(-int(n) // self.bs)
            assert (row[:k] >= 0).all() and (row[k:] == -1).all()
            np.add.at(want, row[:k], 1)
        assert (want == self.refs).all()

    def _take(self, n):
        free = np.flatnonzero(self.refs == 0)
        return None if len(free) < n else [int(x) for x in free[:n]]

    def append(self, rows, counts):
        """Slots of the new tokens, or None (refused)."""
        if len(set(rows)) < len(rows) or any(not 0 <= r < len(self.ctx) for r in rows) or any(c < 0 for c in counts):
            return None
        need = 0
        for r, c in zip(rows, counts):
            end = int(self.ctx[r]) + c
            if end > self.tables.shape[1] * self.bs:
                return None
            if c and self.ctx[r] % self.bs and self.refs[self.tables[r, self.ctx[r] // self.bs]] != 1:
                return None
            need += -(-end // self.bs) - -(-int(self.ctx[r]) // self.bs)
        new = self._take(need)
        if new is None:
            return None
        slots = []
        for r, c in zip(rows, counts):
            for pos in range(int(self.ctx[r]), int(self.ctx[r]) + c):
                if pos % self.bs == 0:
                    page = new.pop(0)
                    self.tables[r, pos // self.bs], self.refs[page] = page, 1
                slots.append(int(self.tables[r, pos // self.bs]) * self.bs + pos % self.bs)
            self.ctx[r] += c
        return slots

    def fork(self, parents, children):
        """False if refused."""
        rows = len(self.ctx)
        if any(not 0 <= r < rows for r in list(parents) + list(children)) or len(set(children)) < len(children) or \
                set(children) & set(parents) or any(self.ctx[c] for c in children):
            return False
        new = self._take(sum(int(self.ctx[p]) % self.bs > 0 for p in parents))
        if new is None:
            return False
        for p, c in zip(parents, children):
            full, rest = divmod(int(self.ctx[p]), self.bs)
            self.tables[c, :full] = self.tables[p, :full]
            self.refs[self.tables[p, :full]] += 1
            if rest:
                src, dst = self.tables[p, full], new.pop(0)
                self.tables[c, full], self.refs[dst] = dst, 1
                for x in self.pages:
                    x[:, dst, :rest] = x[:, src, :rest]
                for x in self.scales:
                    x[:, dst, :, :rest] = x[:, src, :, :rest]
            self.ctx[c] = self.ctx[p]
        return True

    def free(self, rows):
        for r in rows:
            for page in self.tables[r][self.tables[r] >= 0]:
                self.refs[page] -= 1
            self.tables[r], self.ctx[r] = -1, 0

    def compact(self):
        """remap; pages moved away from keep their contents."""
        used, free = np.flatnonzero(self.refs > 0), np.flatnonzero(self.refs == 0)
        U = len(used)
        remap = np.full(len(self.refs), -1, np.int32)
        remap[used] = used
        for src, dst in zip(used[used >= U], free[free < U]):
            remap[src] = dst
            for x in self.pages + self.scales:
                x[:, dst] = x[:, src]
        refs = np.zeros_like(self.refs)
        refs[remap[used]] = self.refs[used]
        live = self.tables >= 0
        self.tables[live] = remap[self.tables[live]]
        self.refs = refs
        return remap
