"""include/gdn_pages.h on lists, one sequence and page after another (no code of the library)."""


class Shared:
    """Lengths, held pages, block table, free stack and page counts of B sequences."""

    def __init__(self, ps, table, free, n_free, lens, held, refs):
        self.ps, self.table, self.lens, self.held, self.refs = ps, [list(r) for r in table], list(lens), list(held), list(refs)
        self.N, self.free, self.n_free = len(free), list(free), n_free
        self.P = len(self.table[0]) if self.table else 1

    def ok(self, g):
        return 0 <= g < self.N

    def fork(self, src, dst, take):
        """(copy_src, copy_dst, status) of the forks; the lists are changed."""
        B, cs, cd, st = len(self.lens), [], [], []
        lens, held, table = list(self.lens), list(self.held), [list(r) for r in self.table]
        named, asked, at = set(), 0, self.n_free
        for s, d, n in zip(src, dst, take):
            cs.append(-1)
            cd.append(-1)
            st.append(32)
            if not (0 <= s < B and 0 <= d < B and s != d and 0 <= n <= lens[s]):
                continue
            full, part = n // self.ps, int(n % self.ps > 0)
            if held[s] > self.P or full + part > held[s] or lens[d] != 0 or held[d] != 0 or d in named:
                continue
            named.add(d)
            asked += part
            if part and asked > self.n_free:
                continue
            st[-1] = 0
            for i in range(full):
                g = table[s][i]
                self.table[d][i] = g
                if self.ok(g):
                    self.refs[g] += 1
                else:
                    st[-1] = 64
            if part:
                at -= 1
                g, f = table[s][full], self.free[at]
                self.table[d][full] = f
                if self.ok(g) and self.ok(f):
                    cs[-1], cd[-1] = g, f
                else:
                    st[-1] = 64
            self.lens[d], self.held[d] = n, full + part
        self.n_free = at
        return cs, cd, st

    def release(self, keep):
        B, cs, cd, st = len(self.lens), [-1] * len(keep), [-1] * len(keep), [0] * len(keep)
        refs = list(self.refs)   # when the call began
        asked, at, given, drops = 0, self.n_free, [], {}
        for b in range(B):
            n, h = keep[b], self.held[b]
            if n < 0 or n > self.lens[b] or h < 0 or h > self.P:
                st[b] = 32
                continue
            need = -(-n // self.ps)
            stay = min(need, h)
            row = self.table[b]
            copy = n % self.ps > 0 and need <= h and self.ok(row[need - 1]) and refs[row[need - 1]] > 0
            asked += copy
            if copy and asked > self.n_free:
                st[b] = 32
                continue
            out = row[stay - copy:h]
            for g in out:
                if self.ok(g):
                    drops[g] = drops.get(g, 0) + 1
                    given.append((g, b))
                else:
                    st[b] |= 64
            if copy:
                at -= 1
                cs[b], cd[b] = row[need - 1], self.free[at]
                row[need - 1] = cd[b]
                if not self.ok(cd[b]):
                    cs[b] = cd[b] = -1
                    st[b] |= 64
            self.lens[b], self.held[b] = n, stay
        pushed, seen = [], set()
        for g, b in given:
            if g not in seen:
                seen.add(g)
                if refs[g] - drops[g] < 0:
                    self.refs[g] = 0
                    pushed.append((g, b))
                else:
                    self.refs[g] = refs[g] - drops[g]
        for g, b in reversed(pushed):
            if at < self.N:
                self.free[at] = g
                at += 1
            else:
                st[b] |= 64
        self.n_free = at
        return cs, cd, st

    def compact(self):
        """(page_map, moves) ; the books are formed anew."""
        count = [0] * self.N
        for row, h in zip(self.table, self.held):
            for g in row[:h]:
                if self.ok(g):
                    count[g] += 1
        used = sum(c > 0 for c in count)
        holes = [g for g in range(used) if count[g] == 0]
        high = [g for g in range(used, self.N) if count[g]][::-1]
        new = [g if c else -1 for g, c in enumerate(count)]
        for a, z in zip(high, holes):
            new[a] = z
        self.refs = [0] * self.N
        for g, c in enumerate(count):
            if c:
                self.refs[new[g]] = c - 1
        for row, h in zip(self.table, self.held):
            row[:h] = [new[g] if self.ok(g) else g for g in row[:h]]
        self.n_free = self.N - used
        self.free[:self.n_free] = range(self.N - 1, used - 1, -1)
        return new, list(zip(high, holes))
