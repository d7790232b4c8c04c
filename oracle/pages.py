"""An allocator that goes row after row, as a host does: what the page calls have to give."""


class Rows:
    """A table: lists of pages and lengths; refs and pools (numpy, first axis the page) are shared."""

    def __init__(self, refs, page_size, pools=()):
        self.refs, self.P, self.pools = refs, page_size, list(pools)
        self.pages, self.lens = [], []

    def need(self, n):
        return -(-n // self.P)

    def new_rows(self, parents, share=None):
        """Rows that begin with the pages of others (-1: empty), the first share positions of them."""
        other = Rows(self.refs, self.P, self.pools)
        for i, p in enumerate(parents):
            n = 0 if p < 0 else self.lens[p]
            if share is not None:
                n = min(n, max(share[i], 0))
            other.pages.append(list(self.pages[p][:self.need(n)]) if p >= 0 else [])
            other.lens.append(n)
            for page in other.pages[-1]:
                self.refs[page] += 1
        return other

    def truncate(self, new_lens=None):
        for s in range(len(self.lens)):
            n = 0 if new_lens is None else min(self.lens[s], max(int(new_lens[s]), 0))
            while len(self.pages[s]) > self.need(n):
                self.refs[self.pages[s].pop()] -= 1
            self.lens[s] = n

    def reserve(self, grow, width):
        """Pages missing, or 0 with every row grown (rows without room stay)."""
        refs, pages, lens = self.refs.copy(), [list(p) for p in self.pages], list(self.lens)
        free = [p for p in range(len(refs)) if refs[p] == 0]
        wanted, moves = 0, []

        def take():
            nonlocal wanted
            wanted += 1
            if wanted > len(free):
                return -1
            refs[free[wanted - 1]] = 1
            return free[wanted - 1]

        for s, n in enumerate(grow):
            n = max(int(n), 0)
            if n == 0 or lens[s] + n > width * self.P:
                continue
            if lens[s] % self.P and refs[pages[s][-1]] > 1:
                old = pages[s][-1]
                refs[old] -= 1
                pages[s][-1] = take()
                moves.append((old, pages[s][-1]))
            while len(pages[s]) < self.need(lens[s] + n):
                pages[s].append(take())
            lens[s] += n
        if wanted > len(free):
            return wanted - len(free)
        self.refs[:] = refs
        self.pages, self.lens = pages, lens
        for src, dst in moves:
            for pool in self.pools:
                pool[dst] = pool[src]
        return 0

    def compact(self):
        """(page_map, pages in use)."""
        used = [p for p in range(len(self.refs)) if self.refs[p] > 0]
        holes = [p for p in range(len(used)) if self.refs[p] == 0]
        to = {p: p for p in used}
        for src, dst in zip([p for p in used if p >= len(used)], holes):
            to[src] = dst
            self.refs[dst], self.refs[src] = self.refs[src], 0
            for pool in self.pools:
                pool[dst] = pool[src]
        self.pages = [[to[p] for p in row] for row in self.pages]
        return [to.get(p, -1) for p in range(len(self.refs))], len(used)
