"""A plain model of a pool of pages: rows of a table, counts, and what each call makes of them."""
import random

import torch

import lossless_float_compression_amd as zx


class Model:
    """Lists on the host; `width` entries a row, those behind a row's pages are kept as they are."""

    def __init__(self, n_pages, T, n, width, seed=0):
        self.n, self.T, self.W, self.rng = n_pages, T, width, random.Random(seed)
        self.refs = [0] * n_pages
        self.held = [0] * n
        self.table = [[self.rng.choice((-5, 0x7FFFFFF0, 3)) for _ in range(width)] for _ in range(n)]

    def pages(self, s):
        return -(-self.held[s] // self.T)

    def fill(self, total):
        """Rows of so many tokens, in pages of their own, shuffled."""
        ids = self.rng.sample(range(self.n), sum(-(-t // self.T) for t in total))
        at = 0
        for s, t in enumerate(total):
            self.held[s] = t
            for j in range(self.pages(s)):
                self.table[s][j] = ids[at]
                self.refs[ids[at]] += 1
                at += 1
        return self

    def fork(self, parents, beams):
        for g in range(len(self.held) // beams):
            par = parents[g * beams:(g + 1) * beams]
            rows = range(g * beams, (g + 1) * beams)
            if any(not -1 <= p < beams for p in par) or any(not 0 <= self.held[r] <= self.W * self.T for r in rows):
                continue
            old = [(self.table[r][:self.pages(r)], self.held[r]) for r in rows]
            for t, _ in old:
                for p in t:
                    self.refs[p] -= 1
            for r, p in zip(rows, par):
                t, h = old[p] if p >= 0 else ([], 0)
                self.held[r] = h
                self.table[r][:len(t)] = t
                for page in t:
                    self.refs[page] += 1

    def trim(self, keep):
        for s, k in enumerate(keep):
            if k < 0 or not 0 <= self.held[s] <= self.W * self.T or k >= self.held[s]:
                continue
            n = self.pages(s)
            self.held[s] = k
            for p in self.table[s][self.pages(s):n]:
                self.refs[p] -= 1

    def extend(self, new, max_q=1 << 30, max_kv=1 << 30):
        """(kv_len, copies, whether there were pages enough)"""
        T = self.T
        ok = [0 <= q <= max_q and 0 <= h and h + q <= min(max_kv, self.W * T) for q, h in zip(new, self.held)]
        goes = []
        for s, q in enumerate(new):
            page = None
            if ok[s] and q > 0 and self.held[s] % T:
                page = self.table[s][self.held[s] // T]
                if not 0 <= page < self.n or self.refs[page] <= 0:
                    ok[s], page = False, None
            goes.append(page)
        refs, copy, taken = list(self.refs), [], 0
        for s, page in enumerate(goes):
            if page is None:
                copy.append(False)
                continue
            writers = [t for t, p in enumerate(goes) if p == page]
            keeps = len(writers) >= self.refs[page] and writers[0] == s
            copy.append(not keeps)
            refs[page] = 1 if len(writers) >= self.refs[page] else self.refs[page] - len(writers)
        need = [-(-(self.held[s] + q) // T) - self.pages(s) + copy[s] if ok[s] and q > 0 else 0 for s, q in enumerate(new)]
        free = [p for p in range(self.n) if self.refs[p] <= 0]
        if sum(need) > len(free):
            return [0] * len(new), [], False
        self.refs = refs
        copies = []
        for s, q in enumerate(new):
            if need[s]:
                first = self.pages(s) - copy[s]
                for j in range(first, first + need[s]):
                    page = free[taken]
                    taken += 1
                    if copy[s] and j == first:
                        copies.append((self.table[s][j], page, self.held[s] % T))
                    self.table[s][j] = page
                    self.refs[page] = 1
            if ok[s]:
                self.held[s] += q
        return [h if o else 0 for h, o in zip(self.held, ok)], copies, True

    def compact(self):
        live = [p for p in range(self.n) if self.refs[p] > 0]
        holes = [p for p in range(len(live)) if self.refs[p] <= 0]
        move = dict(zip([p for p in live if p >= len(live)], holes))
        remap = [-1] * self.n
        for p in live:
            remap[p] = move.get(p, p)
        refs = [0 if x > 0 else x for x in self.refs]
        for p in live:
            refs[remap[p]] = self.refs[p]
        self.refs = refs
        for s in range(len(self.held)):
            for j in range(self.pages(s)):
                self.table[s][j] = remap[self.table[s][j]]
        return [(a, b, self.T) for a, b in move.items()], remap


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Device:
    """The model's state on the GPU, and the calls."""

    def __init__(self, m, cap=None):
        self.m = m
        self.table, self.held, self.kv = i32(m.table), i32(m.held), i32([77] * len(m.held))
        self.pool = zx.PagePool(m.n, m.T, refs=i32(m.refs))
        self.err = i32([0])
        self.copies = zx.PageCopies(max(cap or 0, len(m.held), m.n // 2), device="cuda")

    def batch(self, new, **kw):
        start = [0]
        for q in new:
            start.append(start[-1] + q)
        return zx.PagedBatch(i32(start), self.kv, self.table, **kw)

    def same(self, err=0):
        m = self.m
        assert self.table.tolist() == m.table
        assert self.held.tolist() == m.held
        assert self.pool.refs.tolist() == m.refs
        assert int(self.err) == err
        self.err.zero_()

    def listed(self):
        n = int(self.copies.count)
        rest = self.copies.pairs[n:]
        assert bool((rest == -1).all())              # entries behind the count are not written
        got = [tuple(x) for x in self.copies.pairs[:n].tolist()]
        self.copies.pairs.fill_(-1)
        return got

    def fork(self, parents, beams, err=0, **kw):
        self.pool.fork(self.table, self.held, i32(parents).view(-1, beams), err=self.err, **kw)
        self.m.fork(parents, beams)
        self.same(err)

    def trim(self, keep, err=0, **kw):
        self.pool.trim(self.table, self.held, None if keep is None else i32(keep), err=self.err, **kw)
        self.m.trim([0] * len(self.m.held) if keep is None else keep)
        self.same(err)

    def extend(self, new, err=0, max_q=None, max_kv=None, **kw):
        self.pool.extend(self.batch(new, max_q=max_q, max_kv=max_kv), self.held, copies=self.copies, err=self.err, **kw)
        kv, copies, enough = self.m.extend(new, 1 << 30 if max_q is None else max_q, 1 << 30 if max_kv is None else max_kv)
        assert self.kv.tolist() == kv
        assert self.listed() == copies
        self.same(6 if not enough and not err else err)
        return copies

    def compact(self, err=0, table=True, **kw):
        _, remap = self.pool.compact(*((self.table, self.held) if table else (None, None)), copies=self.copies, err=self.err, **kw)
        copies, want = self.m.compact()
        assert remap.tolist() == want
        assert self.listed() == copies
        self.same(err)
        return copies
