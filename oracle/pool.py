"""Plain model of the device page pool: who holds which page, forks, copies of
shared pages before they are written to, compaction.

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__.py``).

The pages describe a block table whose rollback returns pages to a free list
("Build a Speculative Decoding Engine ...", *Rollback Protocol*).  Readings:
pages are taken lowest number first, by sequence and then by position; a page
held by several sequences is counted, and copied before one of them writes to
it, unless every holder is about to, when the longest (then the lowest-numbered)
keeps it.  A sequence that a reservation gives no slots sits the pass out: its
last page is marked until a reservation serves it.
"""
from __future__ import annotations

SLOTS = 64
OUT = 1 << 26


def pages_for(slots: int) -> int:
    return -(-slots // SLOTS)


class Pool:
    def __init__(self, batch: int, n_pages: int, max_pages: int):
        self.batch, self.n_pages, self.max_pages = batch, n_pages, max_pages
        self.held = [[] for _ in range(batch)]   # pages in position order
        self.len = [0] * batch
        self.guard = [False] * batch             # its partly filled page is not to be written to
        self.out = [set() for _ in range(batch)]  # entries that say that it sits passes out

    def ref(self) -> list:
        r = [0] * self.n_pages
        for row in self.held:
            for p in row:
                r[p] += 1
        return r

    def table(self) -> list:
        out = []
        for row, g, marks, length in zip(self.held, self.guard, self.out, self.len):
            e = list(row)
            if g:
                e[length // SLOTS] = -2 - e[length // SLOTS]
            for i in marks:
                e[i] = -2 - OUT - e[i]
            out.append(e + [-1] * (self.max_pages - len(e)))
        return out

    def sit_out(self, b):
        last = pages_for(self.len[b]) - 1
        if last >= 0:
            self.guard[b] = False
            self.out[b].add(last)

    def reserve(self, n) -> tuple[list, list]:
        """(moves (source, destination, slots), sequences that the free pages did not cover)."""
        by_seq = not isinstance(n, int)
        n = [n] * self.batch if isinstance(n, int) else list(n)
        ok = [self.len[b] + n[b] <= self.max_pages * SLOTS for b in range(self.batch)]
        for b in range(self.batch):
            if ok[b]:
                self.held[b] = self.held[b][:pages_for(self.len[b])]
                self.out[b] = {i for i in self.out[b] if i < len(self.held[b])}
            elif self.len[b] <= self.max_pages * SLOTS:
                self.sit_out(b)
        ref = self.ref()
        writers = {}
        for b in range(self.batch):
            if ok[b] and n[b] and self.len[b] % SLOTS:
                writers.setdefault(self.held[b][-1], []).append(b)
        keeper = {p: max(bs, key=lambda b: (self.len[b] % SLOTS, -b))
                  for p, bs in writers.items() if len(bs) == ref[p]}
        free = [p for p in range(self.n_pages) if ref[p] == 0]
        moves, short, taken = [], [], 0
        for b in range(self.batch):
            if not ok[b]:
                continue
            L, row = self.len[b], self.held[b]
            partial = bool(n[b]) and L % SLOTS > 0
            copy = partial and keeper.get(row[-1]) != b
            c = (pages_for(L + n[b]) - pages_for(L) if n[b] else 0) + copy
            if taken + c > len(free):  # (a later sequence may need less)
                short.append(b)
                self.sit_out(b)
                continue
            if n[b] == 0:
                if by_seq:
                    self.sit_out(b)
                continue
            got = free[taken:taken + c]
            taken += c
            if copy:
                q = got.pop(0)
                moves.append((row[-1], q, L % SLOTS))
                row[-1] = q
            self.guard[b] = False
            self.out[b].discard(len(row) - 1)
            row += got
        return moves, short

    def fork(self, src, dst) -> list:
        """Pairs that were left out."""
        bad = []
        pairs = list(zip(src, dst))
        for i, (a, b) in enumerate(pairs):
            inside = 0 <= a < self.batch and 0 <= b < self.batch
            if not inside or sum(d == b for _, d in pairs) != 1 or any(s == b for s, _ in pairs):
                bad.append(i)
                continue
            self.held[b] = self.held[a][:pages_for(self.len[a])]
            self.len[b] = self.len[a]
            self.out[b] = self.out[a] & {len(self.held[b]) - 1}
            self.guard[b] = self.len[a] % SLOTS > 0 and not self.out[b]
            if self.guard[b]:
                self.guard[a] = True
        return bad

    def free(self, seqs):
        for b in seqs:
            if 0 <= b < self.batch:
                self.held[b], self.len[b], self.guard[b], self.out[b] = [], 0, False, set()

    def compact(self) -> list:
        ref = self.ref()
        used = [p for p in range(self.n_pages) if ref[p]]
        u = len(used)
        moves = list(zip([p for p in used if p >= u], [p for p in range(u) if ref[p] == 0]))
        to = dict(moves)
        self.held = [[to.get(p, p) for p in row] for row in self.held]
        return moves
