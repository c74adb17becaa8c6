"""Seeded 4-bit caches for the tests of the gdn_kv4.h calls."""

from __future__ import annotations

import numpy as np
import torch

import gated_deltanet_speculative_amd as gdn
from oracle import kv4_oracle as K
from round_util import Paged, as_numpy, dev


class Paged4(Paged):
    """Paged, with random 4-bit caches: codes of every kind, scales within 2^spread of each other."""

    def __init__(self, C, N, Hq, Hkv, D, page, dtype, lens, seed=0, layers=0, spread=3, **kw):
        super().__init__(C, N, Hq, Hkv, 64, 1, dtype, [0] * C, seed=seed, **kw)  # (its caches are not used)
        del self.k, self.v
        rng, sh = self.rng, self.sh
        need = [-(-(n + N) // page) for n in lens]
        n_pages, max_pages = sum(need) + 2, max(need)
        ids = rng.permutation(n_pages)
        self.table, self.len = np.full((sh.n_slots, max_pages), -1, np.int32), np.zeros(sh.n_slots, np.int32)
        at = 0
        for c in range(C):
            self.table[self.slots[c], :need[c]] = ids[at:at + need[c]]
            self.len[self.slots[c]] = lens[c]
            at += need[c]
        self.sh = sh._replace(head_dim=D, page_size=page, n_pages=n_pages, max_pages=max_pages)
        lead = (layers,) if layers else ()
        shape = (*lead, n_pages, Hkv, page)
        codes = lambda: rng.integers(0, 256, (*shape, D // 2)).astype(np.uint8)  # noqa: E731
        scales = lambda: rng.integers(126 - spread, 126, (*shape, D // 32)).astype(np.uint8)  # noqa: E731
        self.host = [codes(), scales(), codes(), scales()]
        self.cache = gdn.Kv4Cache(*(dev(a) for a in self.host))

    def values(self):
        """The caches' values, as the call's dtype holds them."""
        k, v = (K.values(self.host[j], self.host[j + 1]) for j in (0, 2))
        if self.sh.dtype is torch.float16:
            k, v = k.astype(np.float16).astype(np.float64), v.astype(np.float16).astype(np.float64)
        return k, v

    def pull(self):
        """The device's arrays."""
        return [as_numpy(t) for t in self.cache]

    def push(self):
        for t, a in zip(self.cache, self.host):
            t.copy_(torch.from_numpy(a))

    def place(self, c, t):
        """Page and place of row t of lane c."""
        return int(self.table[self.slots[c], t // self.sh.page_size]), t % self.sh.page_size
