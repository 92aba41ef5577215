"""A plain model of the pages of a paged cache: the four operators one row and one entry
after another, on lists. Test infrastructure only."""


def pages_of(n, bs):
    return -(-n // bs)


class Pages:
    """The state (ref, table, lens) and, per page, a list of what its positions hold."""

    def __init__(self, num_blocks, rows, max_blocks, bs):
        self.ref, self.lens, self.bs = [0] * num_blocks, [0] * rows, bs
        self.table = [[-1] * max_blocks for _ in range(rows)]
        self.data = [[None] * bs for _ in range(num_blocks)]

    def fork(self, parents, children, fork_len=None):
        for i, (p, c) in enumerate(zip(parents, children)):
            n = self.lens[p] if fork_len is None else fork_len[i]
            for j in range(pages_of(n, self.bs)):
                self.table[c][j] = self.table[p][j]
                self.ref[self.table[p][j]] += 1
            self.lens[c] = n

    def extend(self, rows, new_len):
        """False, with nothing changed, if the pool has too few free pages."""
        free = [p for p, n in enumerate(self.ref) if n == 0]
        keep = ([*self.ref], [*self.lens], [[*r] for r in self.table], [[*d] for d in self.data])
        try:
            for r, n in zip(rows, new_len):
                old = self.lens[r]
                j, fill = divmod(old, self.bs)
                if fill and n > old and self.ref[self.table[r][j]] > 1:
                    src, dst = self.table[r][j], free.pop(0)
                    self.data[dst][:fill] = self.data[src][:fill]
                    self.ref[src] -= 1
                    self.ref[dst] = 1
                    self.table[r][j] = dst
                for j in range(pages_of(old, self.bs), pages_of(n, self.bs)):
                    self.table[r][j] = free.pop(0)
                    self.ref[self.table[r][j]] = 1
                self.lens[r] = n
        except IndexError:
            self.ref, self.lens, self.table, self.data = keep
            return False
        return True

    def trim(self, rows, new_len):
        for r, n in zip(rows, new_len):
            for j in range(pages_of(n, self.bs), pages_of(self.lens[r], self.bs)):
                self.ref[self.table[r][j]] -= 1
                self.table[r][j] = -1
            self.lens[r] = n

    def compact(self):
        """(remap, L)"""
        live = sum(1 for n in self.ref if n)
        holes = [p for p in range(live) if self.ref[p] == 0]
        remap = [p if n else -1 for p, n in enumerate(self.ref)]
        for p in range(live, len(self.ref)):
            if self.ref[p]:
                h = remap[p] = holes.pop(0)
                self.ref[h], self.ref[p] = self.ref[p], 0
                self.data[h] = [*self.data[p]]
        for r, n in enumerate(self.lens):
            for j in range(pages_of(n, self.bs)):
                self.table[r][j] = remap[self.table[r][j]]
        return remap, live

    def content(self, r):
        return [self.data[self.table[r][j // self.bs]][j % self.bs] for j in range(self.lens[r])]

    def check(self):
        want = [0] * len(self.ref)
        for r, n in enumerate(self.lens):
            for j in range(pages_of(n, self.bs)):
                want[self.table[r][j]] += 1
        assert want == self.ref
