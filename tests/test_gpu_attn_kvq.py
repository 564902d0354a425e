"""Attention over the 4-bit cache on the GPU against its 64-bit form over what the cache
stands for.

Tolerances, as for the 16-bit cache.  Codes times scales are exact in fp16; a weight is
rounded to fp16, the result to q's type t (h(t)); scores are fp32 sums of d products (off
by ds = d 2^-24 scale max_j sum |q k_j|, a weight by 2 ds): |o - ref| <= h(t) |ref| +
(2^-11 + 2 ds + 2^-16) A + 2^-33 B, with A = sum p |v| and 2^-16 for the exponential, the
sums and the joining of parts.  B = sum |v| stands for the small weights: a row's largest
is 2^8 at least in fp16, whose steps end at 2^-24, so a weight below 2^-14 is off by half
of that, 2^-33 of the largest, which the sum of all weights is not below.  (Values that
are exactly 0 where the large weights are leave nothing but that: they are common here.)"""
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


class Attn4:
    """One attention call's device tensors."""

    def __init__(self, cache, q, ctx, new, parents, dtype, scale, q_pad=0, max_tokens=None):
        N, self.hq, d = q.shape
        self.dm = G.AttnDims.make_kvq(len(new), int(sum(new)), max_tokens or max([1, *new]), self.hq, cache.h_kv, cache.d,
                                      G.GDN_BF16 if dtype == torch.bfloat16 else G.GDN_FP16, cache.n_pages, cache.page_size,
                                      cache.table.shape[1], *cache.strides)
        self.qs = self.hq * d + q_pad
        buf = torch.full((max(N, 1), self.qs), float("nan"), dtype=dtype)
        buf[:N, :self.hq * d] = q.reshape(N, -1)
        self.q, self.k, self.v = buf.cuda(), cache.k.cuda(), cache.v.cuda()
        self.units = cache.units
        self.table, self.ctx, self.off = i32(cache.table), i32(ctx), i32(offsets(new))
        self.par = i32([x for p in parents for x in p]) if parents else None
        self.o = torch.full((max(N, 1), self.hq, d), float("nan"), dtype=dtype, device="cuda")
        n = G.gdn_attention_kvq_workspace_bytes(self.dm)
        self.ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")   # NaN everywhere
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.scale, self.N = scale, N

    def __call__(self, stream=None, **kw):
        G.gdn_paged_attention_kvq(self.dm, self.q, self.qs, self.k, self.v, *self.units, self.table, self.ctx, self.off, self.par,
                                  self.scale, self.o, self.ws, self.ws.numel(), self.status, stream=stream, **kw)

    def out(self):
        self()
        torch.cuda.synchronize()
        return self.o.cpu()[:self.N]


def case(seed, dtype, d, hq, hkv, page, layout, units, ctx, new, tree, q_std=1.0):
    rng = np.random.default_rng(seed)
    cache = Q.make_cache4(rng, [a + b for a, b in zip(ctx, new)], hkv, d, page, layout, units)
    g = torch.Generator().manual_seed(seed)
    q = (torch.randn((sum(new), hq, d), generator=g) * q_std).to(dtype)
    parents = [R.random_tree(rng, k) if k else [] for k in new] if tree else None
    return cache, q, parents


def sum_of_values(cache, ctx, new, hq):
    """B: [N][h_q][d], over all of a token's sequence."""
    rows = [cache.view(cache.v, s, c + n).nan_to_num().abs().sum(0).repeat_interleave(hq // cache.h_kv, 0).expand(n, -1, -1)
            for s, (c, n) in enumerate(zip(ctx, new))]
    return torch.cat(rows)


def check(o, ref, A, B, big, dtype, d):
    ds = d * 2.0 ** -24 * big
    tol = R.half_step(dtype) * ref.abs() + (2.0 ** -11 + 2 * ds + 2.0 ** -16) * A + 2.0 ** -33 * B + 1e-30
    err = ((o.double() - ref).abs() / tol)
    assert torch.isfinite(o).all()
    print(f"largest error / tolerance {float(err.max()):.3f}")
    assert float(err.max()) <= 1.0


CASES = [
    # dtype, d, hq, hkv, page, layout, units, ctx, new, tree
    ("bf16", 256, 16, 2, 16, "dense", (1, 1), [0], [1], False),                          # the first token of all
    ("bf16", 256, 16, 2, 16, "heads", (0.5, 4), [1, 63, 64, 65, 200], [1] * 5, False),   # single tokens around a tile's end
    ("fp16", 128, 32, 8, 16, "dense", (1, 1), [7, 127, 128, 300], [1] * 4, False),
    ("bf16", 64, 8, 8, 8, "padded", (2, 0.25), [5, 130], [1, 1], False),
    ("bf16", 256, 16, 2, 32, "dense", (1, 1), [40, 0, 100, 63], [16, 7, 0, 16], True),    # trees, an empty sequence
    ("fp16", 256, 12, 2, 8, "padded", (1, 1), [33, 500], [33, 64], True),                # group of 6: 64 nodes are 384 rows
    ("bf16", 128, 20, 4, 64, "heads", (1, 1), [90, 10, 1], [40, 3, 64], True),            # group of 5
    ("fp16", 64, 6, 6, 128, "dense", (1, 1), [17, 129], [64, 1], True),
    ("bf16", 256, 16, 2, 64, "dense", (0.125, 1), [100], [77], False),                   # a prompt's chunk
    ("bf16", 256, 4, 4, 16, "padded", (1, 1), [0, 50], [200, 1], False),                  # group of 1: 128 tokens a tile
    ("fp16", 128, 8, 2, 256, "dense", (1, 1), [0, 31, 0, 5], [130, 1, 0, 65], False),     # mixed, odd, an empty one
    ("fp16", 64, 16, 2, 1024, "heads", (1, 8), [3], [150], False),
    ("bf16", 128, 128, 1, 16, "dense", (1, 1), [70], [3], True),                          # group of 128: a token is a tile
    ("bf16", 256, 24, 4, 16, "dense", (1, 1), [1500, 3], [5, 2], False),                  # long and short beside each other
    ("fp16", 256, 16, 2, 16, "dense", (1, 1), [700, 9, 0, 64], [2, 2, 1, 2], True),       # rows of several tokens, few of them
    ("bf16", 128, 8, 8, 32, "padded", (1, 1), [257, 31], [9, 5], True),                   # group of 1, few tokens
    ("bf16", 64, 10, 2, 16, "dense", (1, 1), [333, 0, 12], [3, 1, 2], False),
]


@pytest.mark.parametrize("k", range(len(CASES)))
def test_attention(k):
    name, d, hq, hkv, page, layout, units, ctx, new, tree = CASES[k]
    dtype = R.DTYPES[name]
    cache, q, parents = case(100 + k, dtype, d, hq, hkv, page, layout, units, ctx, new, tree)
    ref, A, big = R.attention(q.double(), cache, ctx, new, parents, d ** -0.5)
    a = Attn4(cache, q, ctx, new, parents, dtype, d ** -0.5, q_pad=8 * (k % 3))
    o = a.out()
    assert int(a.status) == 0
    check(o, ref, A, sum_of_values(cache, ctx, new, hq), big, dtype, d)


@pytest.mark.parametrize("d,new", [(256, 3), (256, 40), (128, 1), (128, 40), (64, 7)])
@pytest.mark.parametrize("std", [1e-25, 1e-3, 8.0])
def test_flat_and_peaked(std, d, new):
    """Nearly equal scores, and scores that make one position take all; the running maximum moves along the context.
    bf16 rows of very different sizes."""
    dtype = torch.bfloat16
    cache, q, _ = case(7, dtype, d, 8, 2, 32, "dense", (1, 1), [900], [new], False, q_std=std)
    up = torch.linspace(0.1, 3.0, 900 + new)
    for x in range(900 + new):                       # later keys are larger
        cache.put(cache.k, 0, x, cache.rows(cache.k, 0, x, 1.0) * up[x], 1.0)
    q = (q.double() * torch.logspace(0, 2 if std < 1 else 0, q.shape[0] * q.shape[1], dtype=torch.float64).view(q.shape[0], -1, 1)).to(dtype)
    ref, A, big = R.attention(q.double(), cache, [900], [new], None, d ** -0.5)
    a = Attn4(cache, q, [900], [new], None, dtype, d ** -0.5)
    o = a.out()
    assert int(a.status) == 0
    check(o, ref, A, sum_of_values(cache, [900], [new], 8), big, dtype, d)


@pytest.mark.parametrize("d,hq,n", [(256, 16, 16), (256, 8, 3), (128, 8, 16), (64, 2, 7), (128, 4, 2)])
def test_nan_stays_where_it_is_seen(d, hq, n):
    """NaN blocks of nodes reach the rows that see them, in their 16 columns for values, and no others."""
    dtype, hkv, ctx = torch.float16, 2, 70
    cache, q, par = case(11, dtype, d, hq, hkv, 16, "dense", (1, 1), [ctx], [n], True)
    clean = Q.Cache4(cache.k.clone(), cache.v.clone(), cache.table, cache.page_size, cache.n_pages, cache.strides, hkv, d, cache.units)
    ref, A, big = R.attention(q.double(), clean, [ctx], [n], par, d ** -0.5)
    node = n - 1
    cache.v[cache.scales_at(0, ctx + node)[1, 2]] = 0x7f      # head 1, columns 32 .. 47
    a = Attn4(cache, q, [ctx], [n], par, dtype, d ** -0.5)
    o = a.out()
    sees = torch.tensor([node in R.path_of(par[0], i) for i in range(n)])
    want = torch.zeros(n, hq, d, dtype=torch.bool)
    want[sees, hq // 2:, 32:48] = True
    assert torch.equal(torch.isnan(o), want)
    check(torch.where(want, 0.0, o.double()).to(dtype), torch.where(want, 0.0, ref), A, sum_of_values(clean, [ctx], [n], hq), big, dtype, d)
    cache.v[cache.scales_at(0, ctx + node)] = clean.v[clean.scales_at(0, ctx + node)]
    cache.k[cache.scales_at(0, ctx + node)[0, 0]] = 0xff      # a key of head 0: the whole row of those that see it
    o = Attn4(cache, q, [ctx], [n], par, dtype, d ** -0.5).out()
    want[:] = False
    want[sees, :hq // 2] = True
    assert torch.equal(torch.isnan(o), want)
    # in the context everybody sees it
    cache.v[cache.scales_at(0, 3)[1, 0]] = 0x7f
    o = Attn4(cache, q, [ctx], [n], par, dtype, d ** -0.5).out()
    want[:, hq // 2:, 0:16] = True
    assert torch.equal(torch.isnan(o), want)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_nan_in_many_short_sequences(d):
    """As above for a CTA's many segments of one tile, of which several are under way at once."""
    rng = np.random.default_rng(d)
    S, n, hq, hkv = 1600, 7, 8, 2
    ctx, new = [int(x) for x in rng.integers(0, 50, S)], [n] * S
    cache, q, par = case(12, torch.float16, d, hq, hkv, 16, "dense", (1, 1), ctx, new, True)
    want = torch.zeros(S, n, hq, d, dtype=torch.bool)
    for s in range(S):
        node = int(rng.integers(0, n))
        cache.v[cache.scales_at(s, ctx[s] + node)[1, 1]] = 0x7f      # head 1, columns 16 .. 31
        for i in range(n):
            if node in R.path_of(par[s], i):
                want[s, i, hq // 2:, 16:32] = True
    a = Attn4(cache, q, ctx, new, par, torch.float16, d ** -0.5)
    o = a.out()
    assert int(a.status) == 0 and torch.equal(torch.isnan(o).view(S, n, hq, d), want)


@pytest.mark.parametrize("d,new", [(256, [1, 1]), (128, [5, 2]), (256, [16, 20])])
def test_infinite_and_nan_queries(d, new):
    """A row of q that is not finite spoils its own output only."""
    for dtype in (torch.bfloat16, torch.float16):
        cache, q, _ = case(13, dtype, d, 8, 2, 16, "dense", (1, 1), [100, 30], new, False)
        ref, A, big = R.attention(q.double(), cache, [100, 30], new, None, d ** -0.5)
        q[0, 1, 5], q[-1, 6, 0] = float("inf"), float("nan")
        o = Attn4(cache, q, [100, 30], new, None, dtype, d ** -0.5).out()
        bad = torch.zeros(o.shape[:2], dtype=torch.bool)
        bad[0, 1] = bad[-1, 6] = True
        assert not torch.isfinite(o[bad]).any()
        check(torch.where(bad[..., None], 0.0, o.double()).to(dtype), torch.where(bad[..., None], 0.0, ref), A,
              sum_of_values(cache, [100, 30], new, 8), big, dtype, d)


def big_case(seed, dtype, d, hq, hkv, page, ctx, new):
    """A large cache of random codes and scales on the GPU, its values in 64 bits, and the call's tensors."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    need = [-(-(a + b) // page) for a, b in zip(ctx, new)]
    n_pages, width = sum(need) + 1, max(need) + 1
    block = page * d * 9 // 16
    table = torch.full((len(new), width), n_pages + 5, dtype=torch.int32, device="cuda")
    perm, at = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32), 0
    for s, k in enumerate(need):
        table[s, :k] = perm[at:at + k]
        at += k
    pools = []
    for _ in range(2):
        p = torch.randint(0, 256, (n_pages, hkv, block), generator=g, device="cuda", dtype=torch.int32).to(torch.uint8)
        p[..., page * d // 2:] = torch.randint(0x20, 0x36, (n_pages, hkv, page * d // 16), generator=g, device="cuda", dtype=torch.int32).to(torch.uint8)
        pools.append(p)
    q = torch.randn(sum(new), hq, d, generator=g, device="cuda").to(dtype)
    return table, pools, q, n_pages, width


def big_reference(table, pools, q, page, hkv, d, ctx, new, scale, parents=None):
    grid, e4 = Q.E2M1.cuda(), torch.cat([Q.E4M3, torch.tensor([float("nan")], dtype=torch.float64)]).cuda()
    G_ = q.shape[1] // hkv
    o, A, B = (torch.zeros(q.shape, dtype=torch.float64, device="cuda") for _ in range(3))
    big, n = 0.0, 0
    for s, k in enumerate(new):
        L = ctx[s] + k
        x = torch.arange(L, device="cuda")
        pg, at = table[s].long()[x // page], x % page
        rows = []
        for p in pools:
            c = p[..., :page * d // 2].view(-1, hkv, page, d // 2)[pg, :, at].long()
            sc = e4[p[..., page * d // 2:].view(-1, hkv, page, d // 16)[pg, :, at].long() & 127]
            c = torch.stack([c & 15, c >> 4], -1).flatten(-2)
            v = grid[c & 7] * torch.where(c >= 8, -1.0, 1.0)
            rows.append((v.unflatten(-1, (-1, 16)) * sc[..., None]).flatten(-2))       # [L][hkv][d]
        see = x[None] <= ctx[s] + torch.arange(k, device="cuda")[:, None]
        if parents is not None:
            for i in range(k):
                see[i, ctx[s]:] = False
                see[i, [ctx[s] + j for j in R.path_of(parents[s], i)]] = True
        for h in range(q.shape[1]):
            qq, kk, vv = q[n:n + k, h].double(), rows[0][:, h // G_], rows[1][:, h // G_]
            w = (qq @ kk.T * scale).masked_fill(~see, -float("inf")).softmax(1)
            big = max(big, float((qq.abs() @ kk.abs().T).max()) * scale)
            o[n:n + k, h], A[n:n + k, h] = w @ vv, w @ vv.abs()
            B[n:n + k, h] = vv.abs().sum(0)
        n += k
    return o, A, B, big


BIG = [
    # dtype, d, hq, hkv, page, ctx, new, tree
    ("bf16", 256, 16, 2, 16, [5000, 3, 900, 12000, 64, 1], [1] * 6, False),
    ("fp16", 256, 16, 2, 64, [3000] * 24, [16] * 24, True),
    ("bf16", 256, 12, 2, 8, [777, 2000], [2, 1], False),
    ("bf16", 128, 32, 8, 16, [1500, 400, 0, 2999], [300, 701, 129, 1], False),
    ("fp16", 128, 8, 8, 128, [9000, 100], [3, 2], True),
    ("bf16", 64, 16, 4, 32, [4000, 0], [50, 600], False),
    ("fp16", 64, 8, 8, 8, [6000, 70, 3000], [1, 1, 1], False),
    ("bf16", 256, 8, 1, 64, [30000], [1], False),            # one sequence over the whole GPU
    ("bf16", 256, 16, 2, 32, [200] * 400, [1] * 400, False),  # more items than CTAs
    ("fp16", 128, 16, 4, 16, [100 + 7 * i for i in range(200)], [1 + i % 5 for i in range(200)], True),
]


@pytest.mark.parametrize("k", range(len(BIG)))
def test_large(k):
    name, d, hq, hkv, page, ctx, new, tree = BIG[k]
    dtype, scale = R.DTYPES[name], d ** -0.5
    table, pools, q, n_pages, width = big_case(200 + k, dtype, d, hq, hkv, page, ctx, new)
    rng = np.random.default_rng(k)
    par = [R.random_tree(rng, n) for n in new] if tree else None
    dm = G.AttnDims.make_kvq(len(new), sum(new), max(new), hq, hkv, d, G.GDN_BF16 if name == "bf16" else G.GDN_FP16, n_pages, page, width)
    ws = torch.full((G.gdn_attention_kvq_workspace_bytes(dm),), 255, dtype=torch.uint8, device="cuda")
    st, o = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.full_like(q, float("nan"))
    args = (dm, q, hq * d, pools[0], pools[1], 1.0, 1.0, table, i32(ctx), i32(offsets(new)), i32([x for p in par for x in p]) if tree else None, scale)
    G.gdn_paged_attention_kvq(*args, o, ws, ws.numel(), st)
    assert int(st) == 0
    ref, A, B, big = big_reference(table, pools, q, page, hkv, d, ctx, new, scale, par)
    check(o, ref, A, B, big, dtype, d)
    again = torch.full_like(q, 3.0)
    G.gdn_paged_attention_kvq(*args, again, ws, ws.numel(), st)
    assert torch.equal(o, again)                              # results do not depend on timing


def test_device_errors():
    cache, q, par = case(17, torch.bfloat16, 128, 4, 2, 16, "dense", (1, 1), [40, 10], [4, 4], True)
    bad_table = cache.table.copy()
    bad_table[1, 0] = cache.n_pages
    for code, kw in ((G.GDN_DEV_BAD_NODE_OFF, dict(off=i32([0, 4, 9]))), (G.GDN_DEV_BAD_LEN, dict(ctx=i32([40, -1]))),
                     (G.GDN_DEV_BAD_LEN, dict(ctx=i32([40, 16 * cache.table.shape[1] - 3]))), (G.GDN_DEV_BAD_PAGE, dict(table=i32(bad_table))),
                     (G.GDN_DEV_BAD_PAGE, dict(table=i32(-bad_table - 1))), (G.GDN_DEV_BAD_PARENT, dict(par=i32(par[0] + [-1, 0, 2, 1])))):
        a = Attn4(cache, q, [40, 10], [4, 4], par, torch.bfloat16, 128 ** -0.5)
        for name, v in kw.items():
            setattr(a, name, v)
        a.out()
        assert int(a.status) == code, (kw, int(a.status))


@pytest.mark.parametrize("role", [0, 1, 2, 3, 4])
@pytest.mark.parametrize("d", [256, 64])
def test_waits_run_out(d, role):
    """A wait that nothing ends is given up and reported; the next call is sound."""
    cache, q, _ = case(19, torch.bfloat16, d, 16, 2, 16, "dense", (1, 1), [300], [40], False)
    ref, A, big = R.attention(q.double(), cache, [300], [40], None, d ** -0.5)
    a = Attn4(cache, q, [300], [40], None, torch.bfloat16, d ** -0.5)
    G.gdn_test_stall_next_attention(20_000_000, role)
    a.out()
    assert int(a.status) == G.GDN_DEV_TIMEOUT
    a.status.zero_()
    o = a.out()
    assert int(a.status) == 0
    check(o, ref, A, sum_of_values(cache, [300], [40], 16), big, torch.bfloat16, d)


@pytest.mark.parametrize("role", [0, 1, 2, 3, 4])
@pytest.mark.parametrize("d,new", [(256, 1), (128, 2), (64, 1)])
def test_waits_run_out_few_rows(d, new, role):
    cache, q, _ = case(20, torch.bfloat16, d, 16, 2, 16, "dense", (1, 1), [3000], [new], False)
    ref, A, big = R.attention(q.double(), cache, [3000], [new], None, d ** -0.5)
    a = Attn4(cache, q, [3000], [new], None, torch.bfloat16, d ** -0.5)
    G.gdn_test_stall_next_attention(20_000_000, role)
    a.out()
    assert int(a.status) == G.GDN_DEV_TIMEOUT
    a.status.zero_()
    o = a.out()
    assert int(a.status) == 0
    check(o, ref, A, sum_of_values(cache, [3000], [new], 16), big, torch.bfloat16, d)


def test_streams_and_graphs():
    """Another stream, and two captured graphs with workspaces of their own replayed one after the other."""
    cache, q, par = case(23, torch.bfloat16, 256, 16, 2, 16, "dense", (1, 1), [500, 33], [16, 9], True)
    a, b = (Attn4(cache, q, [500, 33], [16, 9], par, torch.bfloat16, 1 / 16) for _ in range(2))
    want = a.out()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    b(stream=s)
    s.synchronize()
    assert torch.equal(b.o.cpu(), want)
    graphs = []
    for x in (a, b):
        x.o.fill_(0)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            x()
        graphs.append(g)
    for _ in range(3):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    assert torch.equal(a.o.cpu(), want) and torch.equal(b.o.cpu(), want) and int(a.status) == 0


def test_graph_of_few_rows_follows_the_lengths():
    """A captured call of single tokens, replayed while the lengths grow page by page, gives what calls give."""
    ctx, new = [500, 33, 0, 64], [1, 1, 1, 1]
    cache, q, _ = case(24, torch.bfloat16, 256, 16, 2, 16, "dense", (1, 1), [700, 233, 200, 264], new, False)
    a, b = (Attn4(cache, q, ctx, new, None, torch.bfloat16, 1 / 16) for _ in range(2))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        b()
    for _ in range(12):
        want = a.out()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(b.o.cpu(), want) and int(a.status) == int(b.status) == 0
        a.ctx += 17
        b.ctx += 17
