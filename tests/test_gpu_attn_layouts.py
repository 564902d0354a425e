"""Memory layouts that the attention layers' entry points take: layers inside the pools."""
import numpy as np
import pytest
import torch

import attn_ref as R
import gated_deltanet_speculative_gdn_gb300 as G

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # collected on CPU machines, never run there
    pytest.skip("needs a CUDA GPU", allow_module_level=True)


def i32(x):
    return torch.tensor(np.asarray(x, dtype=np.int32), device="cuda")


@pytest.mark.parametrize("order", ["lpthd", "plthd", "ptlhd", "pthld", "phltd", "lphtd"])
def test_move_with_layers_anywhere(order):
    """A cache of L layers, pages, tokens, heads and d in any order with d last: what the commit leaves is what the
    copies of the definition leave."""
    d, hkv, page, layers, dtype = 64, 3, 8, 3, torch.bfloat16
    rng = np.random.default_rng(4)
    ctx, new = [5, 0, 21], [12, 0, 30]
    need = [-(-(a + b) // page) for a, b in zip(ctx, new)]
    pages = sum(need) + 1
    size = dict(l=layers, p=pages, t=page, h=hkv, d=d)
    k, v = (torch.randn([size[x] for x in order], generator=torch.Generator().manual_seed(i)).to(dtype) for i in range(2))
    stride = dict(zip(order, k.stride()))
    perm, table, at = rng.permutation(pages), np.full((3, max(need)), pages + 5), 0
    for s, n in enumerate(need):
        table[s, :n] = perm[at:at + n]
        at += n
    parents = [R.random_tree(rng, n) if n else [] for n in new]
    acc = [11, -1, 29]
    back = [order.index(x) for x in "lpthd"]
    want = [t.clone() for t in (k, v)]
    lens = list(ctx)
    for s in (0, 2):
        path = R.path_of(parents[s], acc[s])
        lens[s] += len(path)
        place = lambda x: (int(table[s, x // page]), x % page)
        for t, src in zip(want, (k, v)):
            for j, x in enumerate(path):
                a, b = place(ctx[s] + j), place(ctx[s] + x)
                t.permute(back)[:, a[0], a[1]] = src.permute(back)[:, b[0], b[1]]
    dm = G.AttnDims.make(3, sum(new), max(new), hkv, hkv, d, G.GDN_BF16, pages, page, max(need), stride["p"], stride["t"],
                         stride["h"])
    kg, vg, nl = k.cuda(), v.cuda(), i32([-7] * 3)
    status = i32([0])
    G.gdn_kv_commit(dm, layers, stride["l"], i32(acc), i32([x for p in parents for x in p]),
                    i32(np.concatenate([[0], np.cumsum(new)])), i32(ctx), i32(table), kg, vg, nl, status)
    torch.cuda.synchronize()
    assert int(status) == 0 and nl.tolist() == lens
    assert torch.equal(kg.cpu(), want[0]) and torch.equal(vg.cpu(), want[1])


@pytest.mark.parametrize("case", ["one buffer in place", "one buffer to its end", "into the gaps of another", "k | v | q"])
@pytest.mark.parametrize("norm", [True, False])
def test_append_from_one_buffer(case, norm):
    """q, k and v as columns of one projection's output, in place or beside it: the bits of separate tensors."""
    d, hq, hkv, page, dtype = 64, 6, 2, 8, torch.bfloat16
    rng = np.random.default_rng(1)
    ctx, new = [3, 0, 30], [5, 1, 17]
    N, wq, wk = sum(new), hq * d, hkv * d
    cache = R.make_cache(rng, [a + b for a, b in zip(ctx, new)], hkv, d, page, dtype, garbage=1.0)
    g = torch.Generator(device="cuda").manual_seed(3)
    q, k, v = (torch.randn((N, w), generator=g, device="cuda").to(dtype) for w in (wq, wk, wk))
    w = 1 + 0.1 * torch.randn(d, generator=g, device="cuda") if norm else None
    dm = G.AttnDims.make(3, N, max(new), hq, hkv, d, G.GDN_BF16, cache.n_pages, page, cache.table.shape[1], *cache.strides)
    half = 16
    inv_freq = torch.tensor([1e4 ** (-i / half) for i in range(half)], dtype=torch.float64, device="cuda")
    pos, off, lens, table = i32(rng.integers(0, 5000, (N, 1))), i32(np.concatenate([[0], np.cumsum(new)])), i32(ctx), i32(cache.table)

    def append(qt, qs, kt, ks, vt, vs, qo, qos):
        kp, vp, status = cache.k.cuda(), cache.v.cuda(), i32([0])
        G.gdn_rope_append(dm, qt, qs, kt, ks, vt, vs, w, w, 1e-6, pos, 1, inv_freq, None, 2 * half, 0, off, lens, table, qo, qos,
                          kp, vp, status)
        torch.cuda.synchronize()
        assert int(status) == 0
        return kp, vp

    want_q = torch.empty_like(q)
    want = append(q, wq, k, wk, v, wk, want_q, wq)
    order = (k, v, q) if case == "k | v | q" else (q, k, v)
    row = torch.cat([*order, torch.full((N, wq + 8), 7.0, dtype=dtype, device="cuda")], 1)
    stride, before = row.stride(0), row.clone()
    at, starts = 0, {}
    for t in order:
        starts[id(t)] = at
        at += t.shape[1]
    part = lambda t: row[:, starts[id(t)]:]
    if case == "one buffer to its end":
        out, first = row, at
    elif case == "into the gaps of another":
        out, first = row, at + 8
    else:
        out, first = row, starts[id(q)]
    qt, qs = (q, wq) if case == "into the gaps of another" else (part(q), stride)
    got = append(qt, qs, part(k), stride, part(v), stride, out[:, first:], stride)
    assert torch.equal(out[:, first:first + wq], want_q)
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    rest = torch.ones(row.shape[1], dtype=torch.bool)
    rest[first:first + wq] = False
    assert torch.equal(row[:, rest], before[:, rest])


def test_no_layers_write_nothing():
    dm = G.AttnDims.make(2, 8, 4, 2, 2, 64, G.GDN_BF16, 4, 8, 2)
    pool, nl, status = torch.ones(4 * 8 * 2 * 64, dtype=torch.bfloat16, device="cuda"), i32([-7, -7]), i32([0])
    assert G.gdn_kv_commit(dm, 0, 0, i32([3, 3]), i32([-1, 0, 1, 2] * 2), i32([0, 4, 8]), i32([1, 2]), i32([[0, 1], [2, 3]]), pool,
                           pool.clone(), nl, status) == G.GDN_OK
    torch.cuda.synchronize()
    assert nl.tolist() == [-7, -7] and int(status) == 0 and bool((pool == 1).all())
