"""Long attention calls built on the GPU, their result in 64 bits, and a copy of the
kernel's schedule that says what of it a call reaches."""
from __future__ import annotations

import numpy as np
import torch

import attn_ref as R
import gated_deltanet_speculative_gdn_gb300 as G

TILE, FRONT = 64, 10   # positions of a tile; what an item costs beside its tiles, in tiles


def item_tiles(ctx, new, hkv, group):
    """Tiles of every item in the order of the schedule: sequence, key/value head, row tile."""
    rows, out = 128 // group, []
    for c, n in zip(ctx, new):
        one = [-(-(c + min((j + 1) * rows, n)) // TILE) for j in range(-(-n // rows))]
        out += one * hkv
    return np.array(out, dtype=np.int64)


def reached(ctx, new, hkv, group, ctas=None):
    """Over the CTAs: the most segments and tiles of one, the most tiles of a segment, and how many hold both
    an item's end and another's beginning that go on elsewhere; and the total of units."""
    if ctas is None:
        ctas = torch.cuda.get_device_properties(0).multi_processor_count
    tiles = item_tiles(ctx, new, hkv, group)
    end = np.cumsum(tiles + FRONT)
    total = int(end[-1])
    active = min(ctas, total)
    cut = np.array([total * b // active for b in range(active + 1)], dtype=np.int64)
    first, last = np.searchsorted(end, cut[:-1], side="right"), np.searchsorted(end, cut[1:] - 1, side="right")
    most_seg = most_tiles = longest = both = 0
    for b in range(active):
        seg = []
        for i in range(first[b], last[b] + 1):
            at = end[i] - tiles[i] - FRONT
            lo, hi = max(cut[b] - at, FRONT), max(min(cut[b + 1] - at, tiles[i] + FRONT), FRONT)
            if hi > lo:
                seg.append(hi - lo)
        most_seg, most_tiles = max(most_seg, len(seg)), max(most_tiles, int(sum(seg)))
        longest = max(longest, max(seg, default=0))
        opens = cut[b] > end[first[b]] - tiles[first[b]] - FRONT
        goes_on = cut[b + 1] < end[last[b]]
        both += bool(opens and goes_on and last[b] > first[b])
    return dict(segments=most_seg, tiles=most_tiles, longest=int(longest), both=both, total=total)


class Call:
    """A paged cache and one call's tensors, all on the GPU.  Places without a position hold NaN, table
    entries past a sequence's pages are out of range.  `pages_of` gives each sequence its pages (None: pages
    of its own in random order)."""

    def __init__(self, seed, name, d, hq, hkv, page, ctx, new, tree=False, pages_of=None, n_pages=None, q_std=1.0,
                 table=None):
        self.dtype, self.d, self.hq, self.hkv, self.page = R.DTYPES[name], d, hq, hkv, page
        self.ctx, self.new = [int(x) for x in ctx], [int(x) for x in new]
        rng = np.random.default_rng(seed)
        g = torch.Generator(device="cuda").manual_seed(seed)
        need = [-(-(a + b) // page) for a, b in zip(self.ctx, self.new)]
        if table is not None:
            pages_of = table
        elif pages_of is None:
            n_pages = sum(need) + 2
            perm, at, pages_of = rng.permutation(n_pages), 0, []
            for k in need:
                pages_of.append(perm[at:at + k])
                at += k
        dense = table is not None
        if dense:
            width = table.shape[1]
        else:
            width = max(need) + 1
            table = np.full((len(need), width), n_pages + 1000, dtype=np.int32)
            for s, k in enumerate(need):
                table[s, :k] = pages_of[s][:k]
        self.table = torch.from_numpy(np.ascontiguousarray(table, dtype=np.int32)).cuda()
        shape = (n_pages * page, hkv, d)
        self.k, self.v = (torch.full(shape, float("nan"), dtype=self.dtype, device="cuda") for _ in range(2))
        rows = (torch.arange(n_pages * page, device="cuda") if dense else
                torch.unique(torch.cat([self.rows(s) for s in range(len(need)) if need[s]])))
        for pool in (self.k, self.v):
            for part in rows.split(1 << 16):
                pool[part] = torch.randn((len(part), hkv, d), generator=g, device="cuda").to(self.dtype)
        self.N = sum(self.new)
        self.q = (torch.randn((self.N, hq, d), generator=g, device="cuda") * q_std).to(self.dtype)
        self.parents = [R.random_tree(rng, n) if n else [] for n in self.new] if tree else None
        self.off = np.concatenate([[0], np.cumsum(self.new)]).astype(np.int32)
        i32 = lambda x: torch.tensor(np.asarray(x, dtype=np.int32), device="cuda")
        self.par = i32([x for p in self.parents for x in p]) if tree else None
        self.off_d, self.ctx_d = i32(self.off), i32(self.ctx)
        self.o = torch.full_like(self.q, float("nan"))
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.scale = d ** -0.5
        self.dm = G.AttnDims.make(len(need), self.N, max([1, *self.new]), hq, hkv, d,
                                  G.GDN_BF16 if name == "bf16" else G.GDN_FP16, n_pages, page, width)
        self.ws = torch.full((G.gdn_attention_workspace_bytes(self.dm),), 255, dtype=torch.uint8, device="cuda")

    def rows(self, s, upto=None):
        """Rows of the pools that hold positions 0 .. of sequence s."""
        n = self.ctx[s] + self.new[s] if upto is None else upto
        x = torch.arange(n, device="cuda")
        return self.table[s].long()[x // self.page] * self.page + x % self.page

    def reached(self):
        return reached(self.ctx, self.new, self.hkv, self.hq // self.hkv)

    def __call__(self):
        G.gdn_paged_attention(self.dm, self.q, self.hq * self.d, self.k, self.v, self.table, self.ctx_d, self.off_d,
                              self.par, self.scale, self.o, self.ws, self.ws.numel(), self.status)
        return self.o

    def out(self):
        self.o.fill_(float("nan"))
        self()
        torch.cuda.synchronize()
        assert int(self.status) == 0
        return self.o.clone()

    def seen(self, s):
        """[new][ctx + new] truth values."""
        c, n = self.ctx[s], self.new[s]
        m = torch.ones((n, c + n), dtype=torch.bool, device="cuda")
        if self.parents:
            line = torch.zeros((n, n), dtype=torch.bool)
            for i in range(n):
                line[i, R.path_of(self.parents[s], i)] = True
            m[:, c:] = line.cuda()
        else:
            m[:, c:] = torch.ones((n, n), dtype=torch.bool, device="cuda").tril()
        return m

    def exact(self, s):
        """Sequence s in 64 bits: o, sum p |v| and sum |v|, [new][hq][d] each, and the largest scale * sum |q k|."""
        gr, rows, seen = self.hq // self.hkv, self.rows(s), self.seen(s)
        a, b = int(self.off[s]), int(self.off[s + 1])
        n = b - a
        q = self.q[a:b].double().view(n, self.hkv, gr, self.d).permute(1, 2, 0, 3).reshape(self.hkv, gr * n, self.d)
        k, v = (p[rows].double().transpose(0, 1) for p in (self.k, self.v))   # [hkv][L][d]
        hide = ~seen.repeat(gr, 1)
        x = (q @ k.transpose(1, 2) * self.scale).masked_fill(hide, float("-inf"))
        big = float((q.abs() @ k.abs().transpose(1, 2) * self.scale).masked_fill(hide, 0.0).max())
        p = torch.softmax(x, -1)
        back = lambda t: t.view(self.hkv, gr, n, self.d).permute(2, 0, 1, 3).reshape(n, self.hq, self.d)
        return back(p @ v), back(p @ v.abs()), back((seen.double() @ v.abs()).repeat(1, gr, 1)), big

    def check(self, o, seqs=None, terms=None):
        """Every output within its roundings of the 64-bit result; the largest share of the tolerance used.
        One rounding to the type is half a step h.  Weights and results are rounded once each; a score is off by
        2^-24 of its `terms` products at most (ds), a weight by twice that; sums of 16 positions are added in fp32
        with an error of a whole step (2^-23) at most, n / 16 of them one after the other, in O and in l; 2^-16 for
        the exponential and the joining of parts.  An fp16 weight is 2^8 at least for the largest score, so the step
        below the normal range, 2^-24, is 2^-32 of that, and half of it counts; a result there has that step too."""
        h, worst = R.half_step(self.dtype), 0.0
        for s in seqs if seqs is not None else range(len(self.new)):
            if self.new[s] == 0:
                continue
            ref, A, V, big = self.exact(s)
            ds = (terms or self.d) * 2.0 ** -24 * big
            steps = 2 * (self.ctx[s] + self.new[s]) / 16 * 2.0 ** -23
            tol = h * ref.abs() + (h + 2 * ds + steps + 2.0 ** -16) * A + 1e-30
            if self.dtype == torch.float16:
                tol += 2.0 ** -33 * V + 2.0 ** -25
            got = o[int(self.off[s]):int(self.off[s + 1])].double()
            assert torch.isfinite(got).all(), s
            worst = max(worst, float(((got - ref).abs() / tol).max()))
        print(f"largest error / tolerance {worst:.3f}")
        assert worst <= 1.0
        return worst
