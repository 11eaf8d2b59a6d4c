"""The pages of a cache, kept in plain lists."""
from __future__ import annotations

__all__ = ["Pool"]


class Pool:
    """Rows of page numbers and the uses of each page; free pages are handed out lowest first, all or none."""

    def __init__(self, n_pages: int, n_rows: int, page: int):
        self.refs, self.rows, self.lens, self.page = [0] * n_pages, [[] for _ in range(n_rows)], [0] * n_rows, page

    def _free(self):
        return [i for i, n in enumerate(self.refs) if n == 0]

    def _drop(self, row, keep):
        while len(row) > keep:
            self.refs[row.pop()] -= 1

    def resize(self, lens):
        """Returns n_free."""
        self.lens = list(lens)
        need = [-(-n // self.page) for n in lens]
        for row, n in zip(self.rows, need):
            self._drop(row, n)
        want = [max(0, n - len(row)) for row, n in zip(self.rows, need)]
        free = self._free()
        if sum(want) <= len(free):
            at = 0
            for row, n in zip(self.rows, want):
                for page in free[at:at + n]:
                    row.append(page)
                    self.refs[page] = 1
                at += n
        return len(free) - sum(want)

    def fork(self, src, dst):
        """Returns n_free and the copies that the caches need: (from page, to page, tokens)."""
        for d in dst:
            self._drop(self.rows[d], 0)
            self.lens[d] = 0
        part = [self.lens[s] % self.page for s in src]
        free = self._free()
        left = len(free) - sum(p > 0 for p in part)
        copies = []
        if left >= 0:
            for s, d, p in zip(src, dst, part):
                self.rows[d] = self.rows[s][:self.lens[s] // self.page]
                for page in self.rows[d]:
                    self.refs[page] += 1
                self.lens[d] = self.lens[s]
                if p:
                    page = free.pop(0)
                    copies.append((self.rows[s][len(self.rows[d])], page, p))
                    self.rows[d].append(page)
                    self.refs[page] = 1
        return left, copies
