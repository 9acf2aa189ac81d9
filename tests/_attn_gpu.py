"""A paged cache for the GPU tests of the attention operators: pages and slots
in no order, a page that no slot holds, NaN or a fill wherever no row is."""
from __future__ import annotations

import numpy as np

from tests._gpu import lib, torch_cuda

DT = {"bf16": "bfloat16", "f32": "float32"}


def io_of(io):
    g = lib()
    return g.IO_BF16 if io == "bf16" else g.IO_F32


def rand(rng, shape, io, scale=1.0):
    """Random values of the type, on the host."""
    torch = torch_cuda()
    return torch.from_numpy((rng.standard_normal(shape) * scale).astype(np.float32)).to(getattr(torch, DT[io]))


def f64(t):
    return t.double().cpu().numpy()


def up(v):
    torch = torch_cuda()
    return None if v is None else torch.from_numpy(np.ascontiguousarray(v)).cuda()


def strided(t, off, pad, fill=7.0):
    """The rows of t inside a wider device buffer, `off` columns from its start, and that buffer."""
    torch = torch_cuda()
    wide = torch.full((t.shape[0], off + t.shape[1] + pad), fill, dtype=t.dtype)
    wide[:, off:off + t.shape[1]] = t
    wide = wide.cuda()
    return wide[:, off:off + t.shape[1]], wide


class Cache:
    """k, v, acc, pos (host copies before the call, device tensors) for entries
    of the given row counts; layout "hr" (heads around rows), "rh" (rows around
    heads) or "pad" (rows and heads with gaps)."""

    def __init__(self, rng, lens, hk, d, page, io, layout="hr", fill=float("nan"), sums=True, extra_pages=3,
                 extra_slots=2, max_pages=None, positions=None):
        torch = torch_cuda()
        self.lens_list, self.hk, self.d, self.page, self.io = list(lens), hk, d, page, io
        n = len(self.lens_list)
        need = [-(-m // page) for m in self.lens_list]
        self.n_pages, self.n_slots = sum(need) + extra_pages, n + extra_slots
        self.max_pages = max_pages or max(max(need, default=1), 1)
        order = rng.permutation(self.n_pages)
        self.slots = rng.permutation(self.n_slots)[:n].astype(np.int32)
        # rows of no entry hold a page number that would fault
        self.table = np.full((self.n_slots, self.max_pages), 2 ** 30, np.int32)
        self.lens = np.full(self.n_slots, -1, np.int32)
        at = 0
        for i, m in enumerate(need):
            self.table[self.slots[i], :m] = order[at:at + m]
            self.lens[self.slots[i]] = self.lens_list[i]
            at += m
        dt = getattr(torch, DT[io])
        self.k, self.v = (torch.full((self.n_pages, hk, page, d), fill, dtype=dt) for _ in "kv")
        self.acc = torch.full((self.n_pages, hk, page), fill) if sums else None
        self.pos = torch.full((self.n_pages, hk, page), -7, dtype=torch.int32) if sums else None
        for i, m in enumerate(self.lens_list):
            pg, off = self.where(i)
            self.k[pg, :, off], self.v[pg, :, off] = rand(rng, (m, hk, d), io), rand(rng, (m, hk, d), io)
            if sums:
                self.acc[pg, :, off] = torch.from_numpy(rng.random((m, hk)).astype(np.float32))
                p = np.arange(m) if positions is None else positions(i, m)
                p = np.broadcast_to(np.asarray(p, np.int32).reshape(m, 1), (m, hk))
                self.pos[pg, :, off] = torch.from_numpy(p.copy())
        self.kd, self.vd = self._place(self.k, layout), self._place(self.v, layout)
        self.accd = None if not sums else self.acc.cuda()
        self.posd = None if not sums else self.pos.cuda()
        self.tabled, self.lensd, self.slotsd = up(self.table), up(self.lens), up(self.slots)

    def _place(self, t, layout):
        torch = torch_cuda()
        if layout == "hr":
            return t.cuda()
        if layout == "rh":
            return t.transpose(1, 2).contiguous().cuda().transpose(1, 2)
        gap = torch.full((self.n_pages + 1, self.hk + 1, self.page + 1, self.d + 16), 3.0, dtype=t.dtype).cuda()
        view = gap[:self.n_pages, :self.hk, :self.page, :self.d]
        view.copy_(t)
        return view

    def where(self, i, lo=0, hi=None):
        """Pages and places of the rows lo..hi of entry i."""
        r = np.arange(lo, self.lens_list[i] if hi is None else hi)
        return self.table[self.slots[i]][r // self.page].astype(np.int64), r % self.page

    def kv(self, **over):
        return lib().Kv(**{**dict(k=self.kd, v=self.vd, table=self.tabled, lens=self.lensd, acc=self.accd,
                                  pos=self.posd), **over})

    def rows(self, t, i, h, lo=0):
        """Rows lo.. of entry i and head h of a host tensor, in 64 bits."""
        pg, off = self.where(i, lo)
        return t[pg, h, off].double().numpy()


def same(a, b):
    """Bit for bit (NaN included)."""
    torch = torch_cuda()
    a, b = a.cpu(), b.cpu()
    kind = {1: torch.uint8, 2: torch.int16, 4: torch.int32}[a.element_size()]
    return torch.equal(a.contiguous().view(kind), b.contiguous().view(kind))
