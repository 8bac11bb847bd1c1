"""Pages that sequences share, in plain Python: lists of whole numbers and a list of page contents."""


class Pool:
    def __init__(self, table, refs, lengths, page_size, pages):
        self.table, self.refs, self.lengths = [list(r) for r in table], list(refs), list(lengths)
        self.P, self.pages = page_size, list(pages)

    def is_page(self, x):
        return 0 <= x < len(self.refs)

    def fork(self, parents):
        """Returns whether a parent was out of range."""
        old, ns, B = [list(r) for r in self.table], list(self.lengths), len(self.table)
        for b, q in enumerate(parents):
            if q >= B or q == b:
                continue
            self.table[b] = [-1] * len(old[b]) if q < 0 else list(old[q])
            self.lengths[b] = 0 if q < 0 else ns[q]
        for b in range(B):
            for was, now in zip(old[b], self.table[b]):
                if self.is_page(was):
                    self.refs[was] -= 1
                if self.is_page(now):
                    self.refs[now] += 1
        return any(q >= B for q in parents)

    def reserve(self, counts):
        """Returns (granted, whether a length was out of range)."""
        before, table = list(self.refs), [list(r) for r in self.table]
        free = [x for x in range(len(before)) if before[x] == 0]
        granted, asked, bad, let_go = [], 0, False, []
        for b, (n, c) in enumerate(zip(self.lengths, counts)):
            if n < 0 or n + c > len(table[b]) * self.P:
                granted.append(0)
                bad = True
                continue
            entries = range(n // self.P, -(-(n + c) // self.P)) if c else ()
            want = [e for e in entries if not self.is_page(table[b][e]) or before[table[b][e]] > 1]
            at, asked = asked, asked + len(want)
            if want and asked > len(free):
                granted.append(0)
                continue
            for i, e in enumerate(want):
                was, now = table[b][e], free[at + i]
                if self.is_page(was):
                    let_go.append(was)
                    if e == n // self.P and n % self.P:
                        self.pages[now] = self.pages[was]
                self.table[b][e] = now
                self.refs[now] = 1
            granted.append(c)
        for x in let_go:
            self.refs[x] -= 1
        return granted, bad

    def compact(self):
        used = sum(x != 0 for x in self.refs)
        holes = [x for x in range(used) if self.refs[x] == 0]
        movers = [x for x in range(used, len(self.refs)) if self.refs[x] != 0]
        to = dict(zip(movers, holes))
        for x, y in to.items():
            self.pages[y] = self.pages[x]
            self.refs[y], self.refs[x] = self.refs[x], 0
        self.table = [[to.get(x, x) for x in r] for r in self.table]
        return used
