"""Plain reference of the page operators, on lists and CPU tensors, from their
documentation.  No code of the package."""
import torch

BAD_PAGE, BAD_LEN, NO_PAGE, BAD_PARENT = 1, 2, 8, 16


class Pool:
    """Table (lists, -1: no page), lengths, and the layers' pools
    [layers, 2, pages, kv_heads, page, dim] on the CPU."""

    def __init__(self, table, lens, kv, page):
        self.table, self.lens, self.kv, self.page = [list(r) for r in table], list(lens), kv, page
        self.pages, self.status = kv.shape[2], 0

    def refs(self):
        n = [0] * self.pages
        for row in self.table:
            for p in row:
                if p >= 0:
                    n[p] += 1
        return n

    def need(self, n):
        return -(-n // self.page)

    def count(self):
        for row, n in zip(self.table, self.lens):
            for i, p in enumerate(row):
                if i >= self.need(n):
                    row[i] = -1
                elif not 0 <= p < self.pages:
                    row[i] = -1
                    self.status |= BAD_PAGE

    def fork(self, parents):
        table, lens = [list(r) for r in self.table], list(self.lens)
        for b, p in enumerate(parents):
            if p == -1:
                self.table[b], self.lens[b] = [-1] * len(table[b]), 0
            elif 0 <= p < len(lens):
                self.table[b], self.lens[b] = list(table[p]), lens[p]
            else:
                self.status |= BAD_PARENT

    def resize(self, lens):
        most = len(self.table[0]) * self.page
        for n in lens:
            if not 0 <= n <= most:
                self.status |= BAD_LEN
        lens = [min(max(n, 0), most) for n in lens]
        for row, n in zip(self.table, lens):
            for i in range(self.need(n), len(row)):
                row[i] = -1
        refs = self.refs()
        free = [p for p in range(self.pages) if refs[p] == 0]
        begun = {}
        for b, (row, old, new) in enumerate(zip(self.table, self.lens, lens)):
            if new > old and old % self.page and row[old // self.page] >= 0:
                begun.setdefault(row[old // self.page], []).append(b)
        copies, keeps, missed = [], [], set()
        for b, (row, old, new) in enumerate(zip(self.table, list(self.lens), lens)):
            at, page = old // self.page, None
            if new > old and old % self.page:
                page = row[at] if row[at] >= 0 else None
                if page is None:
                    self.status |= BAD_PAGE
            self.lens[b] = new
            if page is not None and refs[page] > 1 and not (len(begun[page]) == refs[page] and begun[page][0] == b):
                if not free:
                    self.status |= NO_PAGE
                    self.lens[b] = old
                    missed.add(page)
                else:
                    copies.append((page, free[0], old % self.page))
                    row[at] = free.pop(0)
            elif page is not None:
                keeps.append((b, page, old, self.need(old)))
            first = self.need(new)
            while first and row[first - 1] < 0:
                first -= 1
            for i in range(first, self.need(new)):
                if not free:
                    self.status |= NO_PAGE
                    self.lens[b] = min(self.lens[b], i * self.page)
                    break
                row[i] = free.pop(0)
        for b, page, old, held in keeps:      # another still reads the page
            if page in missed:
                self.status |= NO_PAGE
                self.lens[b] = old
                self.table[b][held:] = [-1] * (len(self.table[b]) - held)
        for source, target, slots in copies:
            self.kv[:, :, target, :, :slots] = self.kv[:, :, source, :, :slots]

    def compact(self):
        refs = self.refs()
        used = sum(n > 0 for n in refs)
        holes = [p for p in range(used) if refs[p] == 0]
        top = [p for p in range(self.pages - 1, used - 1, -1) if refs[p] > 0]
        moved = [p if refs[p] else -1 for p in range(self.pages)]
        for source, target in zip(top, holes):
            moved[source] = target
            self.kv[:, :, target] = self.kv[:, :, source]
        self.table = [[moved[p] if p >= 0 else -1 for p in row] for row in self.table]
        return used, moved

    def copy(self, src, dst, to):
        for s, d in zip(src, dst):
            if 0 <= s < self.pages and 0 <= d < to.pages:
                to.kv[:, :, d] = self.kv[:, :, s]
            else:
                self.status |= BAD_PAGE
