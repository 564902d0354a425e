"""Plain 64-bit forms of the attention-layer operators and of the acceptance, and
random paged caches to run them on.  CPU only, numpy / torch float64."""
from __future__ import annotations

import math
from dataclasses import dataclass

import numpy as np
import torch

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


def half_step(t: torch.dtype) -> float:
    """Largest relative error of one rounding to t."""
    return torch.finfo(t).eps / 2


def random_tree(rng, n):
    par = [-1]
    for i in range(1, n):
        par.append(int(rng.integers(0, i)))
    return par


def path_of(par, node):
    p = []
    while node >= 0:
        p.append(node)
        node = par[node]
    return p[::-1]


@dataclass
class Cache:
    """A paged cache in a given layout; k, v are flat 16-bit buffers on the CPU."""
    k: torch.Tensor
    v: torch.Tensor
    table: np.ndarray
    page_size: int
    n_pages: int
    strides: tuple            # page, token, head (elements)
    h_kv: int
    d: int

    def offset(self, s, x):
        return int(self.table[s, x // self.page_size]) * self.strides[0] + (x % self.page_size) * self.strides[1]

    def view(self, buf, s, n):
        """[n][h_kv][d] rows of sequence s as float64."""
        at = torch.tensor([self.offset(s, x) for x in range(n)], dtype=torch.long).view(-1, 1, 1)
        idx = at + torch.arange(self.h_kv).view(1, -1, 1) * self.strides[2] + torch.arange(self.d)
        return buf[idx].double()

    def index(self, s, x):
        return (torch.tensor(self.offset(s, x)) + torch.arange(self.h_kv).view(-1, 1) * self.strides[2]
                + torch.arange(self.d))


def make_cache(rng, total, h_kv, d, page_size, dtype, layout="token", garbage=float("nan"), extra=2):
    """A cache for sequences of `total` positions, pages in random order, all places
    without a position filled with `garbage`, and table entries past a sequence's
    pages out of range."""
    need = [-(-t // page_size) for t in total]
    n_pages = sum(need) + extra
    width = max(max(need, default=1), 1) + 1
    if layout == "token":         # [page][token][head][d]
        st = (page_size * h_kv * d, h_kv * d, d)
    elif layout == "head":        # [page][head][token][d]
        st = (page_size * h_kv * d, d, page_size * d)
    else:                         # padded rows
        st = ((page_size * (h_kv * (d + 8) + 16)) + 24, h_kv * (d + 8) + 16, d + 8)
    size = (n_pages - 1) * st[0] + (page_size - 1) * st[1] + (h_kv - 1) * st[2] + d
    perm = rng.permutation(n_pages)
    table = np.full((max(len(total), 1), width), n_pages + 1000, dtype=np.int32)
    at = 0
    for s, k in enumerate(need):
        table[s, :k] = perm[at:at + k]
        at += k
    g = torch.Generator().manual_seed(int(rng.integers(1 << 30)))
    bufs = []
    for _ in range(2):
        b = torch.full((size,), garbage, dtype=torch.float32)
        c = Cache(b, b, table, page_size, n_pages, st, h_kv, d)
        for s, t in enumerate(total):
            for x in range(t):
                b[c.index(s, x)] = torch.randn((h_kv, d), generator=g)
        bufs.append(b.to(dtype))
    return Cache(bufs[0], bufs[1], table, page_size, n_pages, st, h_kv, d)


def seen(ctx, i, par=None):
    """Positions that new token i sees."""
    if par is None:
        return list(range(ctx + i + 1))
    return list(range(ctx)) + [ctx + j for j in path_of(par, i)]


def attention(q, cache, ctx, new, parents, scale):
    """q [N][h_q][d] float64 -> (o, bound weights A = p @ |v|, largest scale * sum |q k|)."""
    N, hq, d = q.shape
    G = hq // cache.h_kv
    o, A, big = torch.zeros_like(q), torch.zeros_like(q), 0.0
    n = 0
    for s, k in enumerate(new):
        if k == 0:
            continue
        kk, vv = cache.view(cache.k, s, ctx[s] + k), cache.view(cache.v, s, ctx[s] + k)
        for i in range(k):
            at = torch.tensor(seen(ctx[s], i, parents[s] if parents else None))
            for h in range(hq):
                key, val = kk[at, h // G], vv[at, h // G]
                x = (key @ q[n, h]) * scale
                big = max(big, float((key.abs() @ q[n, h].abs()).max()) * scale)
                w = torch.exp(x - x.max())
                w = w / w.sum()
                o[n, h] = w @ val
                A[n, h] = w @ val.abs()
            n += 1
    return o, A, big


def rope(x, pos, inv_freq, axis, rot, interleaved, w=None, eps=0.0):
    """x [N][h][d] float64 -> (turned rows, |y_a| + |y_b| per element)."""
    y = x.clone()
    if w is not None:
        y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + eps) * w
    z, mag = y.clone(), y.abs().clone()
    for i in range(rot // 2):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
        # positions times frequency modulo one turn in exact integers
        phi = torch.tensor([math.fmod(float(p) * inv_freq[i], 2 * math.pi) for p in pos[:, axis[i]]], dtype=torch.float64)
        c, s = torch.cos(phi)[:, None], torch.sin(phi)[:, None]
        z[..., a] = y[..., a] * c - y[..., b] * s
        z[..., b] = y[..., b] * c + y[..., a] * s
        mag[..., a] = mag[..., b] = y[..., a].abs() + y[..., b].abs()
    return z, mag


def accept(par, tok, p, q, u, u_next, replacement):
    """One sequence by the definition of rejection sampling, with normalised
    distributions at every step -> (accepted, next token, path length)."""
    n = len(par)
    if n == 0:
        return -1, -1, 0
    cur, depth = 0, 1
    while True:
        P = p[cur].astype(np.float64).copy()
        Q = None if q is None else q[cur].astype(np.float64).copy()
        mass, go = 1.0, None
        first = True
        for x in range(cur + 1, n):
            if par[x] != cur:
                continue
            y = tok[x]
            if Q is None:
                if u[x] * mass < P[y]:
                    go = x
                    break
                mass = max(mass - P[y], 0.0)
                P[y] = 0.0
                continue
            if mass <= 0:
                break
            have = P if first else P / P.sum()
            want = Q / mass
            if float(u[x]) * want[y] < have[y]:
                go = x
                break
            P = np.maximum(have - want, 0.0)
            first = False
            if not replacement:
                mass = max(mass - Q[y], 0.0)
                P[y] = 0.0
                Q[y] = 0.0
        if go is None:
            if not P.sum() > 0:
                P = p[cur].astype(np.float64)
            c = np.cumsum(P)
            t = int(np.searchsorted(c, float(u_next) * c[-1], side="right"))
            return cur, min(t, len(P) - 1), depth
        cur, depth = go, depth + 1
