"""Plain 64-bit forms of the 4-bit cache's operators, written from the formats'
definitions, and random 4-bit caches to run them on.  CPU only, torch float64."""
from __future__ import annotations

from dataclasses import dataclass

import numpy as np
import torch

# the formats' non-negative values in ascending order; a value's index is its code
E2M1 = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64)
E4M3 = torch.tensor([(8 + f if e else f) * 2.0 ** (max(e, 1) - 10) for e in range(16) for f in range(8)][:127], dtype=torch.float64)


def nearest_code(grid, x):
    """Index of the value nearest to each x >= 0 (inf: the last); a tie goes to the even index."""
    mid = (grid[1:] + grid[:-1]) / 2
    i = torch.searchsorted(mid, x.contiguous(), right=False)
    tie = (i < len(mid)) & (mid[i.clamp(max=len(mid) - 1)] == x)
    return torch.where(tie & (i % 2 == 1), i + 1, i)


def quantise(x, unit):
    """[..., d] -> codes [..., d / 2], scales [..., d / 16], uint8."""
    x = x.double().unflatten(-1, (-1, 16))
    fine = torch.isfinite(x).all(-1)
    y = torch.where(fine[..., None], x, 0.0) / unit
    si = nearest_code(6 * E4M3, y.abs().amax(-1))            # the borders of max / 6, times 6
    s = E4M3[si]
    code = nearest_code(E2M1, torch.where(s[..., None] > 0, y.abs() / s[..., None], 0.0))
    # (a sign where the element has one, and a scale: the stored codes of zeros keep it)
    code = code + torch.where((s[..., None] > 0) & torch.signbit(y), 8, 0)
    code = torch.where(fine[..., None], code, 0).flatten(-2).to(torch.uint8)
    scale = torch.where(fine, si, 0x7f).to(torch.uint8)
    return code[..., 0::2] | code[..., 1::2] << 4, scale


def values(codes, scales, unit):
    c = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).long()
    x = E2M1[c & 7] * torch.where(c >= 8, -1.0, 1.0)
    s = torch.where((scales & 0x7f) == 0x7f, float("nan"), E4M3[(scales & 0x7f).long().clamp(max=126)])
    s = s * torch.where(scales >= 128, -1.0, 1.0)
    return (x.unflatten(-1, (-1, 16)) * s[..., None] * unit).flatten(-2)


@dataclass
class Cache4:
    """A 4-bit paged cache; k, v are flat byte buffers on the CPU (one buffer for both when interleaved)."""
    k: torch.Tensor
    v: torch.Tensor
    table: np.ndarray
    page_size: int
    n_pages: int
    strides: tuple            # page, head (bytes)
    h_kv: int
    d: int
    units: tuple

    def _index(self, s, x, per, base):
        """[h_kv][per] byte indices of the row of position x (codes: base 0)."""
        page, at = int(self.table[s, x // self.page_size]), x % self.page_size
        return (page * self.strides[0] + base + at * per + torch.arange(self.h_kv).view(-1, 1) * self.strides[1]
                + torch.arange(per))

    def codes_at(self, s, x):
        return self._index(s, x, self.d // 2, 0)

    def scales_at(self, s, x):
        return self._index(s, x, self.d // 16, self.page_size * self.d // 2)

    def put(self, buf, s, x, rows, unit):
        c, sc = quantise(rows, unit)
        buf[self.codes_at(s, x)], buf[self.scales_at(s, x)] = c, sc

    def rows(self, buf, s, x, unit):
        """[h_kv][d] float64."""
        return values(buf[self.codes_at(s, x)], buf[self.scales_at(s, x)], unit)

    def view(self, buf, s, n):
        """[n][h_kv][d] rows of sequence s as float64."""
        unit = self.units[0] if buf is self.k else self.units[1]
        if n == 0:
            return torch.zeros(0, self.h_kv, self.d, dtype=torch.float64)
        return torch.stack([self.rows(buf, s, x, unit) for x in range(n)])


def make_cache4(rng, total, h_kv, d, page_size, layout="dense", units=(1.0, 1.0), garbage=0xff, extra=2, std=1.0):
    """A cache for sequences of `total` positions, pages in random order, all bytes of no position `garbage` (0xff:
    codes of -6 with a scale that is NaN), table entries past a sequence's pages out of range."""
    need = [-(-t // page_size) for t in total]
    n_pages = sum(need) + extra
    width = max(max(need, default=1), 1) + 1
    block = page_size * d * 9 // 16
    st = {"dense": (h_kv * block, block), "heads": (block, n_pages * block), "padded": (h_kv * (block + 32) + 48, block + 32)}[layout]
    size = (n_pages - 1) * st[0] + (h_kv - 1) * st[1] + block
    perm = rng.permutation(n_pages)
    table = np.full((max(len(total), 1), width), n_pages + 1000, dtype=np.int32)
    at = 0
    for s, k in enumerate(need):
        table[s, :k] = perm[at:at + k]
        at += k
    g = torch.Generator().manual_seed(int(rng.integers(1 << 30)))
    c = Cache4(*(torch.full((size,), garbage, dtype=torch.uint8) for _ in range(2)), table, page_size, n_pages, st, h_kv, d, units)
    for buf, unit in ((c.k, units[0]), (c.v, units[1])):
        for s, t in enumerate(total):
            for x in range(t):
                c.put(buf, s, x, torch.randn((h_kv, d), generator=g) * std * unit, unit)
    return c
