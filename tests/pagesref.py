"""Plain reference of the page accounts: one sequence and one place after the other."""
import numpy as np


class Accounts:
    """Table, pages held, holders of each page and the stack of free ones."""

    def __init__(self, table, held, refs, free, count):
        self.table, self.held, self.refs = table.copy(), held.copy(), refs.copy()
        self.free, self.count = free.copy(), int(count)
        self.bad_seq = self.bad_pos = self.bad_page = self.no_page = False

    @classmethod
    def empty(cls, num_seqs, max_pages, num_pages):
        return cls(np.full((num_seqs, max_pages), -1, np.int32), np.zeros(num_seqs, np.int32),
                   np.zeros(num_pages, np.int32), np.arange(num_pages, dtype=np.int32)[::-1],
                   num_pages)

    def inside(self, page):
        return 0 <= page < len(self.refs)

    def fork(self, src, dst, lens):
        before, held, S = self.table.copy(), self.held.copy(), len(self.held)
        for i, (a, b, n) in enumerate(zip(src, dst, lens)):
            if not (0 <= a < S and 0 <= b < S) or b in dst[:i] or a in dst or held[b] != 0:
                self.bad_seq = True
                continue
            if n < 0 or (n + 63) // 64 > held[a]:
                self.bad_pos = True
                continue
            for j in range((n + 63) // 64):
                page = self.table[b, j] = before[a, j]
                if self.inside(page):
                    self.refs[page] += 1
                else:
                    self.bad_page = True
            self.held[b] = (n + 63) // 64

    def resize(self, keep, room):
        """Returns the pairs to copy [num_seqs, 2]."""
        S, P = self.table.shape
        copies = np.full((S, 2), -1, np.int32)
        before, have_free, taken = self.refs.copy(), self.count, 0
        demand_before, drops = 0, []
        for s in range(S):
            k, n, h = int(keep[s]), int(room[s]), int(self.held[s])
            need = (n + 63) // 64
            if k < 0 or n < k or need > P or h < 0 or h > P or (k + 63) // 64 > h:
                self.bad_pos = True
                continue
            take, drop = [], []  # places, ascending
            for j in range(k // 64, max(h, need)):
                page = self.table[s, j]
                if j >= h:
                    take.append(j)
                elif not self.inside(page):
                    self.bad_page = True
                    if j >= need:
                        drop.append(j)
                elif j >= need:
                    drop.append(j)
                elif before[page] > 1:
                    take.append(j)
                    drop.append(j)
            demand_before += len(take)
            if take and demand_before > have_free:
                self.no_page = True
                continue
            fresh = {j: self.free[have_free - 1 - taken - i] for i, j in enumerate(take)}
            for j in drop:
                drops.append(int(self.table[s, j]))
                if j in fresh and j * 64 < k:
                    copies[s] = drops[-1], fresh[j]
                self.table[s, j] = -1
            for j in take:
                self.table[s, j] = fresh[j]
                self.refs[fresh[j]] = 1
            taken += len(take)
            self.held[s] = need
        drops = [p for p in drops if self.inside(p)]
        for p in drops:
            self.refs[p] -= 1
        self.count -= taken
        last = {p: i for i, p in enumerate(drops)}
        for i, p in enumerate(drops):
            if self.refs[p] == 0 and last[p] == i:
                self.free[self.count] = p
                self.count += 1
        return copies

    def check(self):
        """Every page is free once or held as often as it is counted."""
        S, P = self.table.shape
        held = np.zeros(len(self.refs), int)
        for s in range(S):
            for j in range(self.held[s]):
                held[self.table[s, j]] += 1
            assert (self.table[s, self.held[s]:] == -1).all()
        assert (held == self.refs).all()
        assert sorted(self.free[:self.count]) == list(np.flatnonzero(held == 0))
