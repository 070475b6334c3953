"""CPU model of the paged decode cache's page upkeep, and inputs of the packed
and paged tests.

PagedModel restates, with plain loops over rows and pages, what
cca_paged_reserve, cca_paged_fork and cca_paged_compact do to tables, counts
and lengths, and which pages' contents they move.
"""

from __future__ import annotations

import numpy as np


def window_start(t: int, g: int, w: int) -> int:
    return max(t - w, 0) // g * g


class PagedModel:
    def __init__(self, B, g, w, page, core_pages, raw_pages, core_cols, raw_cols):
        self.B, self.g, self.w, self.page = B, g, w, page
        self.pages = (core_pages, raw_pages)
        self.cols = (core_cols, raw_cols)
        self.table = [np.full((B, n), -1, np.int32) for n in self.cols]
        self.ref = [np.zeros(n, np.int32) for n in self.pages]
        self.lens = np.zeros(B, np.int64)
        # what each page of each pool holds (any label; copies carry it over)
        self.content = [[None] * n for n in self.pages]

    # columns [lo, hi) that a row of n tokens uses, and whether the last one
    # is partly filled
    def used(self, pool, n):
        if n == 0 or (pool == 0 and self.cols[0] == 0):
            return 0, 0, False
        rows = n // self.g if pool == 0 else n
        lo = 0 if pool == 0 else window_start(n - 1, self.g, self.w) // self.page
        return lo, -(-rows // self.page), rows % self.page != 0

    def longest(self):
        raw = self.cols[1] * self.page
        if self.cols[0] == 0:
            return raw
        return min(raw, self.cols[0] * self.page * self.g + self.g - 1)

    def free(self, pool):
        return [p for p in range(self.pages[pool]) if self.ref[pool][p] == 0]

    def reserve(self, n_new):
        """n_new: tokens of each row, or one number for the rows in use.
        Returns the rows that were refused."""
        each = [int(n_new) if x else 0 for x in self.lens] if np.isscalar(n_new) else n_new
        free = [self.free(0), self.free(1)]
        taken, refused, given_back = [0, 0], [], []
        for b, n in enumerate(each):
            if n == 0:
                continue
            if n < 0 or self.lens[b] + n > self.longest():
                refused.append(b)
                continue
            old, new = int(self.lens[b]), int(self.lens[b]) + int(n)
            cols = []
            for pool in (0, 1):
                lo, hi, _ = self.used(pool, new)
                cols.append(range(max(self.used(pool, old)[1], lo), hi))
            at = list(taken)
            for pool in (0, 1):
                taken[pool] += len(cols[pool])
            if any(len(c) and taken[p] > len(free[p]) for p, c in enumerate(cols)):
                refused.append(b)
                continue
            for pool in (0, 1):
                for i, c in enumerate(cols[pool]):
                    p = free[pool][at[pool] + i]
                    self.table[pool][b, c] = p
                    self.ref[pool][p] = 1
            olo, ohi, _ = self.used(1, old)
            for c in range(olo, min(ohi, self.used(1, new)[0])):
                given_back.append(self.table[1][b, c])
                self.table[1][b, c] = -1
            self.lens[b] = new
        for p in given_back:
            self.ref[1][p] -= 1
        return refused

    def fork(self, parent):
        """Returns (rows freed for want of pages, rows whose parent is out of
        range)."""
        wrong = [b for b, p in enumerate(parent) if not -1 <= p < self.B]
        par = [b if b in wrong else int(p) for b, p in enumerate(parent)]
        table, lens = [t.copy() for t in self.table], self.lens.copy()
        old_t, old_n = [t.copy() for t in self.table], self.lens.copy()
        heir = {}  # the row that gets a parent's open pages themselves
        for b, p in enumerate(par):
            if p >= 0 and p not in heir:
                heir[p] = p if par[p] == p else b
        copies = ([], [])
        for b, p in enumerate(par):
            if p == b:
                continue
            for pool in (0, 1):
                table[pool][b] = old_t[pool][p] if p >= 0 else -1
                if p >= 0 and self.used(pool, int(old_n[p]))[2] and heir[p] != b:
                    col = self.used(pool, int(old_n[p]))[1] - 1
                    copies[pool].append((b, col, int(old_t[pool][p, col])))
                    table[pool][b, col] = -1
            lens[b] = old_n[p] if p >= 0 else 0
        self.table, self.lens = table, lens
        self._count()
        failed = set()
        for pool in (0, 1):
            for (b, col, src), p in zip(copies[pool], self.free(pool)):
                self.table[pool][b, col] = p
                self.content[pool][p] = self.content[pool][src]
            failed |= {b for b, col, _ in copies[pool] if self.table[pool][b, col] < 0}
        for b in failed:
            self.lens[b] = 0
            for pool in (0, 1):
                self.table[pool][b] = -1
        self._count()
        return sorted(failed), wrong

    def compact(self):
        live = []
        for pool in (0, 1):
            n = int((self.ref[pool] > 0).sum())
            live.append(n)
            src = [p for p in range(n, self.pages[pool]) if self.ref[pool][p] > 0]
            dst = [p for p in range(n) if self.ref[pool][p] == 0]
            to = dict(zip(src, dst))
            for s, d in to.items():
                self.ref[pool][d], self.ref[pool][s] = self.ref[pool][s], 0
                self.content[pool][d] = self.content[pool][s]
            self.table[pool] = np.vectorize(lambda p: to.get(int(p), int(p)), otypes=[np.int32])(
                self.table[pool]).reshape(self.table[pool].shape)
        return live

    def _count(self):
        for pool in (0, 1):
            t = self.table[pool]
            self.ref[pool] = np.bincount(t[t >= 0], minlength=self.pages[pool]).astype(np.int32)

    def check(self):
        """What holds after every call: counts are the tables' entries; a row
        has a page in exactly its used columns; the page it writes next is
        its own."""
        for pool in (0, 1):
            t = self.table[pool]
            want = np.bincount(t[t >= 0], minlength=self.pages[pool])
            assert np.array_equal(want, self.ref[pool]), ("counts", pool)
            for b in range(self.B):
                lo, hi, open_ = self.used(pool, int(self.lens[b]))
                cols = np.nonzero(t[b] >= 0)[0]
                assert cols.tolist() == list(range(lo, hi)), ("columns", pool, b)
                if open_:
                    assert self.ref[pool][t[b, hi - 1]] == 1, ("open page", pool, b)


def packed_inputs(lens, Hq, Hkv, d, seed, lead=0, trail=0):
    """Bit patterns Q [Hq, total, d], K, V [Hkv, total, d] and offsets of
    sequences with `lead` rows before and `trail` rows behind them."""
    from long_context_sparse_cca_b200 import synth
    total = lead + sum(lens) + trail
    q = synth.random_bf16((Hq, total, d), seed)
    k = synth.random_bf16((Hkv, total, d), seed + 1, scale=1.5)
    v = synth.random_bf16((Hkv, total, d), seed + 2)
    cu = lead + np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    return q, k, v, cu.astype(np.int32)
