"""A book of pages in plain Python, one page at a time: what the calls on the GPU have to arrive at."""
from __future__ import annotations

import numpy as np


class Book:
    """refs, table and lengths, and a cache [layers, pages, page, row] of bytes."""

    def __init__(self, pages, page, rows, width, layers=1, row=16, seed=0):
        rng = np.random.default_rng(seed)
        self.page, self.width = page, width
        self.refs = np.zeros(pages, np.int32)
        self.table = rng.integers(-5, pages + 5, (rows, width)).astype(np.int32)  # what lies behind a row is not read
        self.lens = np.zeros(rows, np.int32)
        self.cache = rng.integers(0, 256, (layers, pages, page, row), dtype=np.uint8)

    def held(self, n):
        return -(-int(n) // self.page)

    def free(self):
        return [int(p) for p in np.flatnonzero(self.refs == 0)]

    def scatter(self, seed=0, keep=0.5):
        """Hold a random part of the free pages from outside, so that what follows is spread out."""
        rng = np.random.default_rng(seed)
        out = np.array([p for p in self.free() if rng.random() < keep], np.int64)
        self.refs[out] += 1
        return out

    def resize(self, new, tokens=0):
        new, old = [int(n) for n in new], [int(n) for n in self.lens]
        for b, (n, o) in enumerate(zip(new, old)):
            for j in range(self.held(n), self.held(o)):
                self.refs[self.table[b, j]] -= 1
        pool, at, out = self.free(), 0, False
        slots = np.full((len(new), tokens), -1, np.int64)
        for b, (n, o) in enumerate(zip(new, old)):
            need = max(0, self.held(n) - self.held(o))
            if need and (out or at + need > len(pool)):
                out, new[b] = True, o
                continue
            for j in range(self.held(o), self.held(o) + need):
                self.table[b, j] = pool[at]
                self.refs[pool[at]] = 1
                at += 1
        for b, (n, o) in enumerate(zip(new, old)):
            for c in range(tokens):
                pos = n - tokens + c
                if pos >= o:
                    slots[b, c] = int(self.table[b, pos // self.page]) * self.page + pos % self.page
        self.lens = np.array(new, np.int32)
        return slots, out

    def fork(self, parents, table_out):
        """The new table and lengths in place of the old ones; whether pages ran out."""
        lens, first, copies = np.zeros(len(parents), np.int32), {}, []
        old = self.refs.copy()
        for r in range(len(self.lens)):  # nobody holds anything
            for j in range(self.held(self.lens[r])):
                old[self.table[r, j]] -= 1
        self.refs = old
        for i, r in enumerate(map(int, parents)):
            if r < 0 or r >= len(self.lens):
                continue
            n = int(self.lens[r])
            lens[i] = n
            for j in range(n // self.page):
                table_out[i, j] = self.table[r, j]
                self.refs[self.table[r, j]] += 1
            if n % self.page:
                if r in first:
                    copies.append((i, r))
                else:
                    table_out[i, n // self.page] = self.table[r, n // self.page]
                    self.refs[self.table[r, n // self.page]] += 1
                first.setdefault(r, i)
        pool, out = self.free(), False
        for k, (i, r) in enumerate(copies):
            n = int(lens[i])
            if k >= len(pool):
                lens[i] = n - n % self.page
                out = True
                continue
            self.cache[:, pool[k], :n % self.page] = self.cache[:, self.table[r, n // self.page], :n % self.page]
            table_out[i, n // self.page] = pool[k]
        for k in range(min(len(pool), len(copies))):
            self.refs[pool[k]] = 1
        self.table, self.lens = table_out, lens
        return out

    def compact(self):
        live = [int(p) for p in np.flatnonzero(self.refs > 0)]
        n = len(live)
        holes = [p for p in range(n) if self.refs[p] == 0]
        moved = [p for p in live if p >= n]
        where = np.full(len(self.refs), -1, np.int32)
        where[live] = live
        for to, frm in zip(holes, moved):
            self.cache[:, to] = self.cache[:, frm]
            self.refs[to], self.refs[frm] = self.refs[frm], 0
            where[frm] = to
        for b, m in enumerate(self.lens):
            h = self.held(m)
            self.table[b, :h] = where[self.table[b, :h]]
        return where, n

    def rows(self, b):
        """What row b's tokens are in the cache, of every layer: [layers, tokens, row]."""
        j = np.arange(int(self.lens[b]))
        return self.cache[:, self.table[b, j // self.page], j % self.page]


class Gpu:
    """The same state on the GPU."""

    def __init__(self, book, extra=0):
        import torch
        import paged_mla_decode_latent_gb300 as mla
        self.mla, self.torch, self.page = mla, torch, book.page
        self.refs, self.lens, self.cache = (torch.from_numpy(x.copy()).cuda() for x in (book.refs, book.lens, book.cache))
        wide = torch.full((book.table.shape[0], book.width + extra), 7, dtype=torch.int32, device="cuda")
        self.table = wide[:, :book.width]
        self.table.copy_(torch.from_numpy(book.table))
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.ws = mla.pages_workspace(len(book.refs), 4 * max(1, book.table.shape[0]))
        self.ws.fill_(0xA5)

    def resize(self, new, tokens=0, **kw):
        t = self.torch
        slots = t.full((self.table.shape[0], tokens), 123, dtype=t.int64, device="cuda") if tokens else None
        self.mla.pages_resize(self.refs, self.table, self.lens, t.tensor([int(n) for n in new], dtype=t.int32, device="cuda"), self.page,
                              self.ws, slots, self.status, **kw)
        return slots

    def fork(self, parents, table_out, **kw):
        t = self.torch
        out = t.from_numpy(table_out.copy()).cuda()
        lens = t.full((len(parents),), 99, dtype=t.int32, device="cuda")
        self.mla.pages_fork(self.refs, self.table, self.lens, t.tensor([int(p) for p in parents], dtype=t.int32, device="cuda"), out, lens,
                            self.cache, self.ws, self.status, **kw)
        self.table, self.lens = out, lens

    def compact(self, **kw):
        t = self.torch
        where, n = t.full_like(self.refs, 55), t.full((1,), 55, dtype=t.int32, device="cuda")
        self.mla.pages_compact(self.refs, self.table, self.lens, self.cache, where, n, self.ws, self.status, **kw)
        return where, n

    def flags(self):
        v = int(self.status)
        self.status.zero_()
        return v

    def same_as(self, book, what=""):
        assert np.array_equal(self.refs.cpu().numpy(), book.refs), what
        assert np.array_equal(self.lens.cpu().numpy(), book.lens), what
        table = self.table.cpu().numpy()
        for b, n in enumerate(book.lens):
            h = book.held(n)
            assert np.array_equal(table[b, :h], book.table[b, :h]), (what, b)
        assert np.array_equal(self.cache.cpu().numpy(), book.cache), what
