"""A plain model of the paged cache's tables (include/dspark.h): Python lists and
sets, one request after the other."""
import numpy as np


class CacheModel:
    def __init__(self, slots, max_pages, pages, page):
        self.S, self.M, self.P, self.page = slots, max_pages, pages, page
        self.rows = [[] for _ in range(slots)]
        self.lens = [0] * slots
        self.refs = [0] * pages

    def free_pages(self):
        return [p for p in range(self.P) if self.refs[p] == 0]

    def fork(self, src, dst):
        status = []
        before = [list(r) for r in self.rows], list(self.lens)
        for i, (s, d) in enumerate(zip(src, dst)):
            bad = (not 0 <= s < self.S or not 0 <= d < self.S or d in dst[:i] or s in dst
                   or len(before[0][d]) > 0)
            status.append(int(bad))
            if not bad:
                # the pages that hold tokens; what s has reserved behind them stays its own
                self.rows[d], self.lens[d] = before[0][s][:-(-before[1][s] // self.page)], before[1][s]
                for p in self.rows[d]:
                    self.refs[p] += 1
        return status

    def reserve(self, add):
        tails = []
        for s in range(self.S):
            t = -1
            if add[s] > 0 and self.lens[s] % self.page and self.lens[s] // self.page < len(self.rows[s]):
                p = self.rows[s][self.lens[s] // self.page]
                t = p if self.refs[p] > 1 else -1
            tails.append(t)
        refs = list(self.refs)
        status, cow = [0] * self.S, [(-1, -1)] * self.S
        free = self.free_pages()
        taken, full = 0, False
        for s in range(self.S):
            if add[s] <= 0:
                continue
            upto = -(-(self.lens[s] + add[s]) // self.page)
            if upto > self.M:
                status[s] = 2
                continue
            p = tails[s]
            # the writer with the most tokens in the page keeps it, if all who share it write
            longest = max((q for q in range(self.S) if tails[q] == p), key=lambda q: (self.lens[q], -q))
            copy = p >= 0 and not (tails.count(p) == refs[p] and longest == s)
            want = max(0, upto - len(self.rows[s])) + copy
            if want and (full or taken + want > len(free)):
                status[s], full = 1, True
                continue
            new = free[taken:taken + want]
            taken += want
            for q in new:
                self.refs[q] = 1
            if copy:
                self.rows[s][self.lens[s] // self.page] = new[0]
                self.refs[p] -= 1
                cow[s] = (p, new[0])
                new = new[1:]
            self.rows[s] += new
        return status, [c[0] for c in cow], [c[1] for c in cow]

    def _cut(self, s, n):
        for p in self.rows[s][n:]:
            self.refs[p] -= 1
        del self.rows[s][n:]

    def commit(self, keep, plus):
        for s in range(self.S):
            if keep[s] != -2 ** 31:
                self.lens[s] = min(max(0, self.lens[s] + keep[s] + plus), len(self.rows[s]) * self.page)
                self._cut(s, -(-self.lens[s] // self.page))

    def free(self, slots):
        for s in slots:
            if 0 <= s < self.S:
                self._cut(s, 0)
                self.lens[s] = 0

    def compact(self):
        used = [p for p in range(self.P) if self.refs[p]]
        n = len(used)
        src, dst = [p for p in used if p >= n], [p for p in range(n) if not self.refs[p]]
        to = dict(zip(src, dst))
        self.rows = [[to.get(p, p) for p in r] for r in self.rows]
        refs = [0] * self.P
        for p in used:
            refs[to.get(p, p)] = self.refs[p]
        self.refs = refs
        return src, dst

    def tables(self):
        table = np.full((self.S, self.M), -1, np.int32)
        for s, r in enumerate(self.rows):
            table[s, :len(r)] = r
        words = np.zeros((self.P + 31) // 32, np.uint32)
        for p in self.free_pages():
            words[p // 32] |= np.uint32(1 << (p % 32))
        return {"table": table, "lens": np.array(self.lens, np.int32),
                "held": np.array([len(r) for r in self.rows], np.int32),
                "refs": np.array(self.refs, np.int32), "free_bits": words.view(np.int32),
                "n_free": np.array([len(self.free_pages())], np.int32)}
