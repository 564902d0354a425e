"""The 4-bit cache's rows on the GPU: quantised into it, read out of it, and moved.

All of it is exact: codes and scales are functions of the 16-bit rows (ties included),
a stored value has 6 significant bits and is a 16-bit value, moves are copies.  So
every comparison is of bits, over the whole buffers."""
import numpy as np
import pytest
import torch

import attn_ref as R
import gated_deltanet_speculative_gdn_gb300 as G
import kv4_ref as Q

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # collected on CPU machines, never run there
    pytest.skip("needs a CUDA GPU", allow_module_level=True)


def i32(x):
    return torch.tensor(np.asarray(x, dtype=np.int32), device="cuda")


def offsets(new):
    return np.concatenate([[0], np.cumsum(new)]).astype(np.int32)


def dims4(cache, new, dtype, hq=None, max_tokens=None):
    return G.AttnDims.make_kvq(len(new), int(sum(new)), max_tokens or max([1, *new]), hq or cache.h_kv, cache.h_kv, cache.d,
                               G.GDN_BF16 if dtype == torch.bfloat16 else G.GDN_FP16, cache.n_pages, cache.page_size,
                               cache.table.shape[1], *cache.strides)


def status():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def rows16(g, n, width, pad, dtype, std=1.0):
    buf = torch.full((n, width + pad), float("nan"), dtype=dtype)
    buf[:, :width] = (torch.randn((n, width), generator=g) * std).to(dtype)
    return buf


CASES = [
    # dtype, d, h_kv, page, layout, units, ctx, new, std, pad
    ("bf16", 256, 2, 16, "dense", (1.0, 1.0), [0], [1], 1.0, 0),
    ("bf16", 256, 2, 32, "heads", (1.0, 0.5), [40, 0, 100, 63], [16, 7, 0, 16], 1.0, 8),
    ("fp16", 128, 3, 8, "padded", (0.25, 2.0), [7, 127, 128, 300], [1, 40, 3, 129], 1.0, 24),
    ("fp16", 64, 1, 1024, "dense", (1.0, 1.0), [1000], [77], 3.0, 0),
    ("bf16", 64, 5, 64, "heads", (2.0 ** -24, 2.0 ** 24), [5, 0], [9, 200], 1.0, 0),     # all saturated, all zeros
    ("bf16", 128, 8, 16, "padded", (1.0, 1.0), [1, 2, 3], [5, 5, 5], 300.0, 8),           # near the largest scale
    ("fp16", 256, 4, 128, "dense", (1.0, 1.0), [0, 9], [33, 300], 0.004, 0),              # scales below the normal ones
]


@pytest.mark.parametrize("k", range(len(CASES)))
def test_append_and_read(k):
    name, d, hkv, page, layout, units, ctx, new, std, pad = CASES[k]
    dtype = R.DTYPES[name]
    rng = np.random.default_rng(k)
    cache = Q.make_cache4(rng, [a + b for a, b in zip(ctx, new)], hkv, d, page, layout, units)
    g = torch.Generator().manual_seed(k)
    N, w = sum(new), hkv * d
    kr, vr = (rows16(g, N, w, pad, dtype, std) for _ in range(2))
    dm = dims4(cache, new, dtype)
    assert G.gdn_kvq_block_bytes(dm) == page * d * 9 // 16
    kp, vp, st = cache.k.cuda(), cache.v.cuda(), status()
    off, ctxt, table = i32(offsets(new)), i32(ctx), i32(cache.table)
    G.gdn_kvq_append(dm, kr.cuda(), w + pad, vr.cuda(), w + pad, *units, off, ctxt, table, kp, vp, st)
    ko, vo = (torch.full((1, N, w + pad), 7.0, dtype=dtype, device="cuda") for _ in range(2))
    G.gdn_kvq_read(dm, 1, 0, kp, vp, *units, off, ctxt, table, ko, vo, w + pad, st)
    torch.cuda.synchronize()
    assert int(st) == 0
    for buf, rows, unit in ((cache.k, kr, units[0]), (cache.v, vr, units[1])):
        n = 0
        for s, m in enumerate(new):
            for i in range(m):
                cache.put(buf, s, ctx[s] + i, rows[n, :w].view(hkv, d), unit)
                n += 1
    assert torch.equal(kp.cpu(), cache.k) and torch.equal(vp.cpu(), cache.v)
    for out, buf, unit in ((ko, cache.k, units[0]), (vo, cache.v, units[1])):
        ref = torch.stack([cache.rows(buf, s, ctx[s] + i, unit) for s, m in enumerate(new) for i in range(m)])
        assert torch.equal(out[0, :, :w].cpu().view(N, hkv, d), ref.to(dtype))   # (overflows to infinity as the type does)
        assert bool((out[0, :, w:] == 7.0).all())


def test_every_value_and_tie():
    """Each block: its largest element a, the others every 16-bit value that is a multiple of a / 96: codes' borders
    among them, for scales that are themselves on borders."""
    for dtype in (torch.bfloat16, torch.float16):
        tops = torch.tensor([6.0, 6.75, 7.125, 6.375, 5.8125, 12.375, 0.05, 1.5 * 2.0 ** -8, 2.0 ** -9, 3 * 2.0 ** -10, 2688, 3000, 4e4, 1e-30, 0.0])
        rows = []
        for a in tops.tolist():
            other = torch.arange(-96, 97) * (a / 96)
            other = torch.cat([other, torch.zeros(-len(other) % 15)]).view(-1, 15)
            rows.append(torch.cat([torch.full((len(other), 1), a), other], 1))
        x = torch.cat(rows).to(dtype)
        x = torch.cat([x, torch.zeros(-len(x) % 4, 16, dtype=dtype)]).view(-1, 64)
        n = len(x)
        cache = Q.make_cache4(np.random.default_rng(0), [n], 1, 64, 16)
        dm = dims4(cache, [n], dtype)
        kp, vp, st = cache.k.cuda(), cache.v.cuda(), status()
        xc = x.cuda()
        G.gdn_kvq_append(dm, xc, 64, -xc, 64, 1.0, 1.0, i32([0, n]), i32([0]), i32(cache.table), kp, vp, st)
        for i in range(n):
            cache.put(cache.k, 0, i, x[i].view(1, 64), 1.0)
            cache.put(cache.v, 0, i, -x[i].view(1, 64), 1.0)
        assert int(st) == 0
        assert torch.equal(kp.cpu(), cache.k) and torch.equal(vp.cpu(), cache.v)


def test_not_finite():
    """One element that is not finite makes its 16 NaN, and no other."""
    for dtype in (torch.bfloat16, torch.float16):
        cache = Q.make_cache4(np.random.default_rng(1), [6], 2, 64, 8)
        x = torch.randn(6, 128, generator=torch.Generator().manual_seed(2)).to(dtype)
        x[0, 3], x[1, 20], x[2, 127], x[4, 64] = float("nan"), float("inf"), -float("inf"), float("nan")
        dm, st = dims4(cache, [6], dtype), status()
        kp, vp = cache.k.cuda(), cache.v.cuda()
        G.gdn_kvq_append(dm, x.cuda(), 128, x.cuda(), 128, 1.0, 1.0, i32([0, 6]), i32([0]), i32(cache.table), kp, vp, st)
        ko, vo = (torch.zeros(6, 128, dtype=dtype, device="cuda") for _ in range(2))
        G.gdn_kvq_read(dm, 1, 0, kp, vp, 1.0, 1.0, i32([0, 6]), i32([0]), i32(cache.table), ko, vo, 128, st)
        for i in range(6):
            cache.put(cache.k, 0, i, x[i].view(2, 64), 1.0)
        assert int(st) == 0 and torch.equal(kp.cpu(), cache.k)
        bad = ~torch.isfinite(x).view(6, -1, 16).all(-1)
        assert torch.equal(torch.isnan(ko.cpu()).view(6, -1, 16).all(-1), bad)
        assert torch.equal(torch.isnan(ko.cpu()).view(6, -1, 16).any(-1), bad)


def test_rows_in_one_buffer():
    """k and v as columns of one buffer, in and out."""
    dtype, d, hkv, n = torch.bfloat16, 64, 2, 21
    cache = Q.make_cache4(np.random.default_rng(3), [n], hkv, d, 8)
    w = hkv * d
    x = torch.randn(n, 2 * w + 16, generator=torch.Generator().manual_seed(4)).to(dtype).cuda()
    out = torch.zeros(n, 2 * w + 16, dtype=dtype, device="cuda")
    dm, st, kp, vp = dims4(cache, [n], dtype), status(), cache.k.cuda(), cache.v.cuda()
    args = (i32([0, n]), i32([0]), i32(cache.table))
    G.gdn_kvq_append(dm, x, 2 * w + 16, x.data_ptr() + 2 * w, 2 * w + 16, 1.0, 1.0, *args, kp, vp, st)
    G.gdn_kvq_read(dm, 1, 0, kp, vp, 1.0, 1.0, *args, out, out.data_ptr() + 2 * w, 2 * w + 16, st)
    assert int(st) == 0
    for i in range(n):
        cache.put(cache.k, 0, i, x[i, :w].cpu().view(hkv, d), 1.0)
        cache.put(cache.v, 0, i, x[i, w:2 * w].cpu().view(hkv, d), 1.0)
        assert torch.equal(out[i, :w].cpu().view(hkv, d).double(), cache.rows(cache.k, 0, i, 1.0))
        assert torch.equal(out[i, w:2 * w].cpu().view(hkv, d).double(), cache.rows(cache.v, 0, i, 1.0))
    assert bool((out[:, 2 * w:] == 0).all())


@pytest.mark.parametrize("d,page,layout,layers,spread", [(256, 16, "dense", 1, False), (128, 8, "padded", 3, False), (64, 64, "heads", 2, True)])
def test_commit(d, page, layout, layers, spread):
    """Accepted paths to the front, for layers one after the other and for layers between the pages."""
    rng = np.random.default_rng(d)
    new, ctx, hkv = [16, 0, 64, 5, 1, 30], [40, 3, 61, 0, 7, 10], 2
    caches = [Q.make_cache4(np.random.default_rng(9), [a + b for a, b in zip(ctx, new)], hkv, d, page, layout) for _ in range(layers)]
    for z, c in enumerate(caches):   # one table for all, other values
        g = torch.Generator().manual_seed(z)
        for buf in (c.k, c.v):
            for s, t in enumerate(a + b for a, b in zip(ctx, new)):
                for x in range(t):
                    c.put(buf, s, x, torch.randn((hkv, d), generator=g), 1.0)
    c0 = caches[0]
    parents = [R.random_tree(rng, k) if k else [] for k in new]
    acc = [int(rng.integers(0, k)) if k else -1 for k in new]
    acc[3] = -1
    parents[2] = [i - 1 for i in range(64)]
    acc[2] = 63                                              # a whole chain: nothing to move
    size = len(c0.k)
    if spread:   # [head][page][layer]: layers lie between the pages
        block = page * d * 9 // 16
        assert c0.strides == (block, c0.n_pages * block)
        def pack(bufs):
            return torch.stack([b.view(hkv, c0.n_pages, block) for b in bufs], 2).reshape(-1).cuda()
        strides, ls = (layers * block, c0.n_pages * layers * block), block
    else:
        pad = (-size) % 16
        def pack(bufs):
            return torch.cat([torch.cat([b, torch.zeros(pad, dtype=torch.uint8)]) for b in bufs]).cuda()
        strides, ls = c0.strides, size + pad
    kp, vp, st = pack([c.k for c in caches]), pack([c.v for c in caches]), status()
    new_len = torch.full((len(new),), -5, dtype=torch.int32, device="cuda")
    dm = G.AttnDims.make_kvq(len(new), sum(new), 64, hkv, hkv, d, G.GDN_BF16, c0.n_pages, page, c0.table.shape[1], *strides)
    G.gdn_kvq_commit(dm, layers, ls, i32(acc), i32([x for p in parents for x in p]), i32(offsets(new)), i32(ctx), i32(c0.table),
                     kp, vp, new_len, st)
    torch.cuda.synchronize()
    assert int(st) == 0
    want = []
    for s, a in enumerate(acc):
        path = R.path_of(parents[s], a)
        want.append(ctx[s] + len(path))
        for c in caches:
            for buf in (c.k, c.v):
                rows = [(buf[c.codes_at(s, ctx[s] + x)].clone(), buf[c.scales_at(s, ctx[s] + x)].clone()) for x in path]
                for j, (co, sc) in enumerate(rows):
                    buf[c.codes_at(s, ctx[s] + j)], buf[c.scales_at(s, ctx[s] + j)] = co, sc
    assert new_len.tolist() == want
    assert torch.equal(kp, pack([c.k for c in caches])) and torch.equal(vp, pack([c.v for c in caches]))


def test_device_errors_write_nothing():
    """Bad lengths, offsets, pages and nodes are reported, and the cache stays as it was."""
    cache = Q.make_cache4(np.random.default_rng(5), [20, 20], 1, 64, 16)
    x = torch.ones(8, 64, dtype=torch.bfloat16, device="cuda")
    dm = dims4(cache, [4, 4], torch.bfloat16)
    kp, vp = cache.k.cuda(), cache.v.cuda()
    out = torch.full((2, 8, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    bad_table = cache.table.copy()
    bad_table[:, 0:2] = cache.n_pages
    far = 16 * cache.table.shape[1] - 3
    for off, ctx, table, code in (([0, 4, 9], [0, 0], cache.table, G.GDN_DEV_BAD_NODE_OFF), ([0, 8, 8], [0, 0], cache.table, G.GDN_DEV_BAD_NODE_OFF),
                                  ([0, 4, 8], [far, far], cache.table, G.GDN_DEV_BAD_LEN), ([0, 4, 8], [-4, -1], cache.table, G.GDN_DEV_BAD_LEN),
                                  ([0, 4, 8], [2 ** 31 - 1, -2 ** 31], cache.table, G.GDN_DEV_BAD_LEN),
                                  ([0, 4, 8], [0, 0], bad_table, G.GDN_DEV_BAD_PAGE), ([0, 4, 8], [0, 0], -bad_table, G.GDN_DEV_BAD_PAGE)):
        if code == G.GDN_DEV_BAD_NODE_OFF:   # (tokens of no sequence are refused one by one; the others are as good as any)
            k2, v2 = kp.clone(), vp.clone()
        else:
            k2, v2 = kp, vp
        st = status()
        G.gdn_kvq_append(dm, x, 64, x, 64, 1.0, 1.0, i32(off), i32(ctx), i32(table), k2, v2, st)
        assert int(st) == code
        st.zero_()
        G.gdn_kvq_read(dm, 1, 0, kp, vp, 1.0, 1.0, i32(off), i32(ctx), i32(table), out[0], out[1], 64, st)
        assert int(st) == code
    assert torch.equal(kp.cpu(), cache.k) and torch.equal(vp.cpu(), cache.v)
    par, new_len = [-1, 0, 1, 2] * 2, torch.full((2,), -5, dtype=torch.int32, device="cuda")
    for off, ctx, table, acc, p, code in (([0, 4, 9], [0, 0], cache.table, [3, 3], par, G.GDN_DEV_BAD_NODE_OFF),
                                          ([0, 4, 8], [0, far], cache.table, [3, 3], par, G.GDN_DEV_BAD_LEN),
                                          ([0, 4, 8], [0, 0], bad_table, [3, 3], par, G.GDN_DEV_BAD_PAGE),
                                          ([0, 4, 8], [0, 0], cache.table, [4, 3], par, G.GDN_DEV_BAD_ACCEPTED),
                                          ([0, 4, 8], [0, 0], cache.table, [3, 3], [-1, 0, 1, 2, -1, 1, 1, 2], G.GDN_DEV_BAD_PARENT)):
        st = status()
        G.gdn_kvq_commit(dm, 1, 0, i32(acc), i32(p), i32(off), i32(ctx), i32(table), kp, vp, new_len, st)
        assert int(st) == code, G.gdn_status_str(code)
    st.fill_(G.GDN_DEV_TIMEOUT)   # after another call's error nothing is written either
    G.gdn_kvq_commit(dm, 1, 0, i32([3, 3]), i32([-1, 0, 0, 0] * 2), i32([0, 4, 8]), i32([0, 0]), i32(cache.table), kp, vp, new_len, st)
    assert new_len.tolist() == [-5, -5]
    assert torch.equal(kp.cpu(), cache.k) and torch.equal(vp.cpu(), cache.v)


def test_far_places_in_a_large_pool():
    """Pages whose bytes lie beyond 2^32 and whose pages are far apart."""
    hkv, d, page = 1, 64, 8
    stride = 1 << 30                                       # bytes between pages
    n_pages = 6
    pool = torch.zeros((n_pages - 1) * stride + 288, dtype=torch.uint8, device="cuda")
    pool2 = torch.zeros_like(pool)
    dm = G.AttnDims.make_kvq(1, 10, 10, hkv, hkv, d, G.GDN_BF16, n_pages, page, 2, stride, 288)
    g = torch.Generator().manual_seed(6)
    x, y = (torch.randn(10, 64, generator=g).bfloat16() for _ in range(2))
    table, st = i32([[5, 4]]), status()
    args = (i32([0, 10]), i32([0]), table)
    G.gdn_kvq_append(dm, x.cuda(), 64, y.cuda(), 64, 1.0, 1.0, *args, pool, pool2, st)
    ko, vo = (torch.zeros(10, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    G.gdn_kvq_read(dm, 1, 0, pool, pool2, 1.0, 1.0, *args, ko, vo, 64, st)
    assert int(st) == 0
    for got, want, p in ((ko, x, pool), (vo, y, pool2)):
        c, sc = Q.quantise(want.view(10, 1, 64), 1.0)
        assert torch.equal(got.cpu().double(), Q.values(c, sc, 1.0).view(10, 64))
        assert torch.equal(p[5 * stride:5 * stride + 256].cpu(), c[:8].flatten())
    new_len = torch.zeros(1, dtype=torch.int32, device="cuda")
    G.gdn_kvq_commit(dm, 1, 0, i32([9]), i32([-1, 0, 0, 0, 0, 0, 0, 0, 0, 0]), *args, pool, pool2, new_len, st)
    G.gdn_kvq_read(dm, 1, 0, pool, pool2, 1.0, 1.0, *args, ko, vo, 64, st)
    assert int(st) == 0 and new_len.tolist() == [2]
    c, sc = Q.quantise(x[9].view(1, 64), 1.0)
    assert torch.equal(ko[1].cpu().double(), Q.values(c, sc, 1.0).view(64))
