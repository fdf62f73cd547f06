"""Fork, free, grow, copy and compact on lists, from the definitions: what the tables, lengths, counts and
pools have to be, for any order of calls."""
import torch


class Book:
    """refs of a pool of pages, and the rules."""

    def __init__(self, num_pages, page):
        self.refs, self.page = [0] * num_pages, page

    def pages(self, n):
        return -(-n // self.page)

    def fork(self, rows, lens, parents):
        new = [list(rows[p][:self.pages(lens[p])]) if p >= 0 else [] for p in parents]
        for row in new:
            for x in row:
                self.refs[x] += 1
        return new, [lens[p] if p >= 0 else 0 for p in parents]

    def free(self, rows, lens, keep=None):
        for b, n in enumerate(lens):
            k = 0 if keep is None else min(n, max(keep[b], 0))
            for x in rows[b][self.pages(k):self.pages(n)]:
                self.refs[x] -= 1
            rows[b] = rows[b][:self.pages(k)]
            lens[b] = k

    def grow(self, rows, lens, news):
        """(copies, left); rows and lens change."""
        spare = [x for x, c in enumerate(self.refs) if c == 0]
        refs, new_rows, copies = list(self.refs), [list(r) for r in rows], [[-1, -1] for _ in lens]
        need = 0
        for b, (n, t) in enumerate(zip(lens, news)):
            row = new_rows[b]
            if t > 0 and n % self.page and refs[row[-1]] > 1:
                refs[row[-1]] -= 1
                copies[b] = [row[-1], spare[need] if need < len(spare) else None]
                row[-1] = copies[b][1]
                need += 1
            while len(row) < self.pages(n + t):
                row.append(spare[need] if need < len(spare) else None)
                need += 1
        left = len(spare) - need
        if left < 0:
            return [[-1, -1] for _ in lens], left
        for x in spare[:need]:
            refs[x] = 1
        self.refs = refs
        rows[:] = new_rows
        for b, t in enumerate(news):
            lens[b] += t
        return copies, left


def table(rows, width, like=None):
    """Rows as a table; entries that no sequence holds are as in `like`, or 0."""
    t = torch.zeros(len(rows), width, dtype=torch.int32) if like is None else like.clone()
    for b, row in enumerate(rows):
        t[b, :len(row)] = torch.tensor(row, dtype=torch.int32)
    return t
