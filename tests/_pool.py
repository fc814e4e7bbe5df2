"""A plain model of a paged cache's pool: Python lists, page by page, with the
error bits that the calls report.  Pages hold distinct random bytes, so a page
that went to the wrong place shows."""
import numpy as np

SLOT, ROW, POOL, REFS = 2, 16, 32, 64


class Pool:
    def __init__(self, num_pages, rows, cols, page_size, page_bytes, seed=0):
        r = np.random.RandomState(seed)
        self.N, self.rows, self.cols, self.P = num_pages, rows, cols, page_size
        self.caches = [r.randint(0, 256, (num_pages, b)).astype(np.uint8) for b in page_bytes]
        self.refs = np.zeros(num_pages, np.int32)
        self.table = np.full((rows, cols), -1, np.int32)
        self.lens = np.zeros(rows, np.int32)
        self.err = 0
        self.rng = r

    def blocks(self, length):
        return -(-int(length) // self.P)

    def fill_row(self, row, length, pages=None):
        """Gives a row `length` tokens on random free pages (or the given ones)."""
        n = self.blocks(length)
        if pages is None:
            pages = self.rng.permutation(np.flatnonzero(self.refs == 0))[:n]
        assert len(pages) == n <= self.cols
        self.table[row, :n] = pages
        for p in pages:
            self.refs[p] += 1
        self.lens[row] = length

    def valid(self, p):
        return 0 <= p < self.N

    def copy(self, src, dst):
        before = [c.copy() for c in self.caches]
        for s, d in zip(src, dst):
            if not (self.valid(s) and self.valid(d)):
                self.err |= SLOT
                continue
            for c, b in zip(self.caches, before):
                c[d] = b[s]

    def fork(self, parents, children):
        lens = self.lens.copy()
        named, todo = set(), []
        for a, ch in zip(parents, children):
            ok = 0 <= a < self.rows and 0 <= ch < self.rows and ch not in named
            ok = ok and lens[a] >= 0 and self.blocks(lens[a]) <= self.cols and lens[ch] == 0
            named.add(ch)
            if ok:
                todo.append((a, ch))
            else:
                self.err |= ROW
        free = [p for p in range(self.N) if self.refs[p] == 0]
        for a, ch in todo:
            whole, part = divmod(int(lens[a]), self.P)
            page = None
            if part:
                if not free:
                    self.err |= POOL
                    continue
                page = free.pop(0)
                self.refs[page] = 1
            for j in range(whole):
                e = int(self.table[a, j])
                if e >= self.N:
                    self.err |= SLOT
                    e = -1
                if e >= 0:
                    self.refs[e] += 1
                self.table[ch, j] = max(e, -1)
            if part:
                self.table[ch, whole] = page
                src = int(self.table[a, whole])
                if self.valid(src):
                    for c in self.caches:
                        c[page] = c[src]
                else:
                    self.err |= SLOT
            self.lens[ch] = lens[a]

    def free(self, rows, window=0, sinks=0):
        for row in rows:
            if not 0 <= row < self.rows:
                self.err |= ROW
                continue
            n = int(self.lens[row])
            blocks = self.blocks(max(n, 0))
            if n < 0 or blocks > self.cols:
                self.err |= ROW
                blocks = min(blocks, self.cols)
            for j in range(blocks):
                first, last = j * self.P, min((j + 1) * self.P, n)  # its tokens
                if window and (first < sinks or last > n - window or (j + 1) * self.P > n):
                    continue
                e = int(self.table[row, j])
                self.table[row, j] = min(e, -1) if e < 0 else -1
                if e < 0:
                    continue
                if e >= self.N:
                    self.err |= SLOT
                elif self.refs[e] <= 0:
                    self.err |= REFS
                else:
                    self.refs[e] -= 1
            if not window:
                self.lens[row] = 0

    def compact(self):
        live = int((self.refs > 0).sum())
        src = [p for p in range(live, self.N) if self.refs[p] > 0]
        dst = [p for p in range(live) if self.refs[p] <= 0]
        for c in self.caches:
            c[dst] = c[src]
        to = dict(zip(src, dst))
        for s, d in to.items():
            self.refs[d], self.refs[s] = self.refs[s], 0
        for row in range(self.rows):
            blocks = self.blocks(max(int(self.lens[row]), 0))
            if self.lens[row] < 0 or blocks > self.cols:
                self.err |= ROW
                blocks = min(blocks, self.cols)
            for j in range(blocks):
                e = int(self.table[row, j])
                if e < live:
                    continue
                if e >= self.N:
                    self.err |= SLOT
                elif e in to:
                    self.table[row, j] = to[e]
                else:
                    self.table[row, j] = -1
                    self.err |= REFS
        return live
