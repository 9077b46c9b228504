"""Paged 8-bit caches for the tests: pools with stale bytes, shuffled pages."""

from __future__ import annotations

import numpy as np

from oracle import cache_ops as co


class Pools:
    """Host and device copies of one cache; the host side runs the oracle."""

    def __init__(self, B, Hkv, d, page, max_pages, seed, spare=2):
        import torch
        rng = np.random.default_rng(seed)
        n = B * max_pages + spare
        self.rng, self.page = rng, page
        self.table = rng.permutation(n)[:B * max_pages].reshape(B, max_pages).astype(np.int32)
        # what a pool holds before its pages are written: any bytes (NaN codes
        # among them), any scale
        self.code = [rng.integers(0, 256, (n, Hkv, page, d), dtype=np.uint8) for _ in range(2)]
        self.scale = [np.exp2(rng.integers(-12, 12, (n, Hkv))).astype(np.float64) for _ in range(2)]
        self.d_table = torch.from_numpy(self.table).cuda()
        self.d_code = [torch.from_numpy(c).cuda() for c in self.code]
        self.d_scale = [torch.from_numpy(s.astype(np.float32)).cuda() for s in self.scale]

    def device(self):
        return self.d_code[0], self.d_code[1], self.d_scale[0], self.d_scale[1], self.d_table

    def fill(self, k, v, lens, counts):
        """The oracle's append on the host copy."""
        for i, x in enumerate((k, v)):
            self.code[i], self.scale[i] = co.cache_append(x, self.code[i], self.scale[i], self.table, lens, counts)

    def upload(self):
        """The host copy to the device (for tests of the readers alone)."""
        import torch
        for i in range(2):
            self.d_code[i].copy_(torch.from_numpy(self.code[i]))
            self.d_scale[i].copy_(torch.from_numpy(self.scale[i].astype(np.float32)))

    def same(self):
        """Is the device cache the host one, byte for byte? (NaN codes of either sign are one.)"""
        for i in range(2):
            c = self.d_code[i].cpu().numpy()
            if not np.array_equal(self.d_scale[i].cpu().numpy().astype(np.float64), self.scale[i]):
                return False
            if not np.array_equal(np.where(c & 127 == 127, 127, c),
                                  np.where(self.code[i] & 127 == 127, 127, self.code[i])):
                return False
        return True


def ints(*v):
    import torch
    return torch.tensor(v, dtype=torch.int32, device="cuda")
