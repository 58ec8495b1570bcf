"""What the calls on page tables do, row by row in plain Python: the reference of the GPU tests, itself tested on the CPU."""


class Tables:
    """rows x width entries (-1: none), lengths, counts; moved: pairs (from, to) of pages copied by the last call."""

    def __init__(self, rows, width, n_pages, ps):
        self.table = [[-1] * width for _ in range(rows)]
        self.lens, self.refs, self.ps, self.width, self.moved = [0] * rows, [0] * n_pages, ps, width, []

    def _held(self, n):
        return -(-n // self.ps)

    def fork(self, parents, children):
        """True where a child was left out."""
        bad, done = False, []
        for i, (p, c) in enumerate(zip(parents, children)):
            if c < 0:
                continue
            R = len(self.lens)
            if c >= R or not 0 <= p < R or c in children[:i] or p in children or self.lens[c] != 0:
                bad = True
            else:
                done.append((p, c))
        for p, c in done:
            for e in range(self._held(self.lens[p])):
                self.table[c][e] = self.table[p][e]
                self.refs[self.table[p][e]] += 1
            self.lens[c] = self.lens[p]
        return bad

    def extend(self, add):
        """False where the free pages did not suffice."""
        self.moved = []
        on = [r for r, a in enumerate(add) if 0 < a <= self.width * self.ps - self.lens[r]]
        part = {r: self.table[r][self.lens[r] // self.ps] for r in on if self.lens[r] % self.ps}
        copied = set()
        for r, x in part.items():
            same = [s for s in part if part[s] == x]
            if len(same) < self.refs[x] or r != min(same):
                copied.add(r)
        need = [(r in copied) + self._held(self.lens[r] + add[r]) - self._held(self.lens[r]) for r in on]
        free = [x for x, k in enumerate(self.refs) if k <= 0]
        if sum(need) > len(free):
            return False
        free = iter(free)
        for r in on:
            n = self._held(self.lens[r])
            if r in copied:
                y = next(free)
                self.moved.append((part[r], y))
                self.refs[part[r]] -= 1
                self.refs[y] = 1
                self.table[r][n - 1] = y
            for e in range(n, self._held(self.lens[r] + add[r])):
                self.table[r][e] = next(free)
                self.refs[self.table[r][e]] = 1
            self.lens[r] += add[r]
        return True

    def free(self, rows, keep=None):
        for i, r in enumerate(rows):
            to = keep[i] if keep else 0
            if r < 0 or self.lens[r] <= to:
                continue
            for e in range(self._held(to), self._held(self.lens[r])):
                self.refs[self.table[r][e]] -= 1
                self.table[r][e] = -1
            self.lens[r] = to

    def compact(self):
        n = len(self.refs)
        live = sum(k > 0 for k in self.refs)
        holes = [x for x in range(live) if self.refs[x] <= 0]
        movers = [x for x in range(live, n) if self.refs[x] > 0]
        remap = [x if k > 0 else -1 for x, k in enumerate(self.refs)]
        self.moved = list(zip(movers, holes))
        for a, b in self.moved:
            remap[a], self.refs[b], self.refs[a] = b, self.refs[a], 0
        for r, k in enumerate(self.lens):
            for e in range(self._held(k)):
                self.table[r][e] = remap[self.table[r][e]]
        return remap

    def check(self, pinned=()):
        """Every count is the number of rows that hold the page (and of others' holds)."""
        want = [0] * len(self.refs)
        for x in pinned:
            want[x] += 1
        for r, k in enumerate(self.lens):
            for e in range(self._held(k)):
                want[self.table[r][e]] += 1
        assert want == self.refs
