"""The attention layers' operators on the GPU against their 64-bit forms.

Tolerances.  One rounding to the 16-bit type t is off by h = eps(t) / 2 of the
value.  Attention rounds each weight and the result once, and forms scores in fp32
(d products and sums, each off by 2^-24 of its terms at most, so a score by
ds = d 2^-24 scale max_j sum |q k_j| and a weight, which has one in its numerator and
one in its denominator, by 2 ds): |o - ref| <= h |ref| + (h + 2 ds + 2^-16) A, with
A = sum p |v| and 2^-16 for the exponential, the sums and the joining of parts.
Rotary rounds once; before it come at most 16 fp32 roundings and an angle
good to 2^-22: |z - ref| <= h |ref| + 2^-19 (|y_a| + |y_b|).  Moves are exact."""
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


def offsets(new):
    return np.concatenate([[0], np.cumsum(new)]).astype(np.int32)


def gdims(cache, new, hq, dtype, max_tokens=None):
    return G.AttnDims.make(len(new), int(sum(new)), max_tokens or max([1, *new]), hq, cache.h_kv, cache.d,
                           G.GDN_BF16 if dtype == torch.bfloat16 else G.GDN_FP16, cache.n_pages, cache.page_size,
                           cache.table.shape[1], *cache.strides)


class Attn:
    """One attention call's device tensors."""

    def __init__(self, cache, q, ctx, new, parents, dtype, scale, q_pad=0, max_tokens=None):
        N, self.hq, d = q.shape
        self.dm = gdims(cache, new, self.hq, dtype, max_tokens)
        self.qs = self.hq * d + q_pad
        buf = torch.full((max(N, 1), self.qs), float("nan"), dtype=dtype)
        buf[:N, :self.hq * d] = q.reshape(N, -1)
        self.q, self.k, self.v = buf.cuda(), cache.k.cuda(), cache.v.cuda()
        self.table, self.ctx, self.off = i32(cache.table), i32(ctx), i32(offsets(new))
        self.par = i32([x for p in parents for x in p]) if parents else None
        self.o = torch.full((max(N, 1), self.hq, d), float("nan"), dtype=dtype, device="cuda")
        n = G.gdn_attention_workspace_bytes(self.dm)
        self.ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")   # NaN everywhere
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.scale, self.N = scale, N

    def __call__(self, stream=None, **kw):
        G.gdn_paged_attention(self.dm, self.q, self.qs, self.k, self.v, self.table, self.ctx, self.off, self.par, self.scale,
                              self.o, self.ws, self.ws.numel(), self.status, stream=stream, **kw)

    def out(self):
        self()
        torch.cuda.synchronize()
        return self.o.cpu()[:self.N]


def case(seed, dtype, d, hq, hkv, page, layout, ctx, new, tree, q_std=1.0):
    rng = np.random.default_rng(seed)
    cache = R.make_cache(rng, [a + b for a, b in zip(ctx, new)], hkv, d, page, dtype, layout)
    g = torch.Generator().manual_seed(seed)
    q = (torch.randn((sum(new), hq, d), generator=g) * q_std).to(dtype)
    parents = [R.random_tree(rng, k) if k else [] for k in new] if tree else None
    return cache, q, parents


def check(o, ref, A, big, dtype, d):
    h = R.half_step(dtype)
    ds = d * 2.0 ** -24 * big
    tol = h * ref.abs() + (h + 2 * ds + 2.0 ** -16) * A + 1e-30
    err = ((o.double() - ref).abs() / tol)
    assert torch.isfinite(o).all()
    print(f"largest error / tolerance {float(err.max()):.3f}")
    assert float(err.max()) <= 1.0


CASES = [
    # dtype, d, hq, hkv, page, layout, ctx, new, tree
    ("bf16", 256, 16, 2, 16, "token", [0], [1], False),                        # the first token of all
    ("bf16", 256, 16, 2, 16, "token", [1, 63, 64, 65, 200], [1] * 5, False),   # single tokens around a tile's end
    ("fp16", 128, 32, 8, 16, "token", [7, 127, 128, 300], [1] * 4, False),
    ("bf16", 64, 8, 8, 8, "head", [5, 130], [1, 1], False),
    ("bf16", 256, 16, 2, 32, "token", [40, 0, 100, 63], [16, 7, 0, 16], True),  # trees, an empty sequence
    ("fp16", 256, 12, 2, 8, "padded", [33, 500], [33, 64], True),              # group of 6: 64 nodes are 384 rows
    ("bf16", 128, 20, 4, 64, "head", [90, 10, 1], [40, 3, 64], True),          # group of 5
    ("fp16", 64, 6, 6, 128, "token", [17, 129], [64, 1], True),
    ("bf16", 256, 16, 2, 64, "token", [100], [77], False),                     # a prompt's chunk
    ("bf16", 256, 4, 4, 16, "padded", [0, 50], [200, 1], False),               # group of 1: 128 tokens a tile
    ("fp16", 128, 8, 2, 256, "token", [0, 31, 0, 5], [130, 1, 0, 65], False),  # mixed, odd, an empty one
    ("fp16", 64, 16, 2, 1024, "head", [3], [150], False),
    ("bf16", 128, 128, 1, 16, "token", [70], [3], True),                       # group of 128: a token is a tile
    ("bf16", 256, 24, 4, 16, "token", [1500, 3], [5, 2], False),               # long and short beside each other
]


@pytest.mark.parametrize("k", range(len(CASES)))
def test_attention(k):
    name, d, hq, hkv, page, layout, ctx, new, tree = CASES[k]
    dtype = R.DTYPES[name]
    cache, q, parents = case(100 + k, dtype, d, hq, hkv, page, layout, ctx, new, tree)
    ref, A, big = R.attention(q.double(), cache, ctx, new, parents, d ** -0.5)
    a = Attn(cache, q, ctx, new, parents, dtype, d ** -0.5, q_pad=8 * (k % 3))
    o = a.out()
    assert int(a.status) == 0
    check(o, ref, A, big, dtype, d)


@pytest.mark.parametrize("std", [1e-3, 8.0])
def test_attention_flat_and_peaked(std):
    """Nearly equal scores, and scores that make one position take all; the running
    maximum moves along the context."""
    dtype, d = torch.bfloat16, 256
    cache, q, parents = case(7, dtype, d, 16, 2, 16, "token", [700], [16], True, q_std=std)
    ref, A, big = R.attention(q.double(), cache, [700], [16], parents, d ** -0.5)
    check(Attn(cache, q, [700], [16], parents, dtype, d ** -0.5).out(), ref, A, big, dtype, d)


@pytest.mark.parametrize("name,d,hq,hkv", [("fp16", 128, 8, 2), ("bf16", 256, 16, 2), ("fp16", 256, 6, 3), ("bf16", 64, 4, 4)])
@pytest.mark.parametrize("step", [0.02, 0.1])
def test_attention_rising_scores(name, d, hq, hkv, step):
    """Keys grow along the context, so the maximum rises from tile to tile, by a little or by much."""
    dtype = R.DTYPES[name]
    cache, q, _ = case(8, dtype, d, hq, hkv, 16, "token", [600], [2], False)
    for x in range(602):
        at = cache.index(0, x)
        cache.k[at] = (cache.k[at].float() * step * x).abs().to(dtype)
    q = q.abs()
    ref, A, big = R.attention(q.double(), cache, [600], [2], None, d ** -0.5)
    check(Attn(cache, q, [600], [2], None, dtype, d ** -0.5).out(), ref, A, big, dtype, d)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("tree", [True, False])
@pytest.mark.parametrize("d,hq,hkv", [(256, 16, 2), (128, 4, 2), (64, 4, 4)])
def test_what_is_not_seen_has_no_influence(bad, tree, d, hq, hkv):
    """One new token's key and value are not finite: the rows that do not see it
    keep their results bit for bit, the rows that see it are not finite where its
    value is not."""
    dtype = torch.bfloat16
    ctx, new = [70, 20], [40, 24]
    cache, q, parents = case(9, dtype, d, hq, hkv, 16, "token", ctx, new, tree)
    clean = Attn(cache, q, ctx, new, parents, dtype, d ** -0.5).out()
    where = 11
    cache.v[cache.index(0, ctx[0] + where)[:, 3:5]] = bad
    dirty = Attn(cache, q, ctx, new, parents, dtype, d ** -0.5).out()
    sees = [i for i in range(new[0]) if ctx[0] + where in R.seen(ctx[0], i, parents[0] if parents else None)]
    rest = [n for n in range(sum(new)) if n not in sees]
    assert 0 < len(sees) < new[0]
    assert torch.equal(clean[rest], dirty[rest])
    assert not torch.isfinite(dirty[sees][:, :, 3:5]).any()
    others = [c for c in range(d) if c not in (3, 4)]
    assert torch.equal(clean[sees][:, :, others], dirty[sees][:, :, others])
    # a key that is not finite: the same rows keep theirs
    cache.v[cache.index(0, ctx[0] + where)[:, 3:5]] = 0.5
    cache.k[cache.index(0, ctx[0] + where)] = bad
    dirty = Attn(cache, q, ctx, new, parents, dtype, d ** -0.5).out()
    clean_v = Attn(cache, q, ctx, new, parents, dtype, d ** -0.5)
    assert torch.isfinite(dirty[rest]).all()
    cache.k[cache.index(0, ctx[0] + where)] = 0.25
    assert torch.equal(Attn(cache, q, ctx, new, parents, dtype, d ** -0.5).out()[rest], dirty[rest])
    assert clean_v.N == sum(new)


def test_nan_in_the_context_reaches_the_rows_that_see_it():
    dtype, d = torch.bfloat16, 128
    cache, q, _ = case(10, dtype, d, 8, 2, 16, "token", [100, 100], [3, 3], False)
    cache.v[cache.index(1, 50)[0, :1]] = float("nan")
    o = Attn(cache, q, [100, 100], [3, 3], None, dtype, d ** -0.5).out()
    assert torch.isfinite(o[:3]).all() and torch.isnan(o[3:, :4, 0]).all() and torch.isfinite(o[3:, 4:]).all()


@pytest.mark.parametrize("d,hq,hkv,name", [(256, 16, 2, "bf16"), (128, 8, 2, "fp16"), (64, 4, 2, "bf16")])
@pytest.mark.parametrize("where", [range(100, 101), range(64, 128), range(128, 320)])
def test_nan_keys_in_the_context_reach_the_rows_that_see_them(d, hq, hkv, name, where):
    """One key, a whole tile of keys and several: the sequence's rows are NaN at that key/value head, in
    whichever parts of the work the keys fall; the other sequence's and the other heads' are not."""
    dtype = R.DTYPES[name]
    cache, q, _ = case(14, dtype, d, hq, hkv, 16, "token", [700, 100], [2, 2], False)
    for x in where:
        cache.k[cache.index(0, x)[0]] = float("nan")
    o = Attn(cache, q, [700, 100], [2, 2], None, dtype, d ** -0.5).out()
    assert torch.isnan(o[:2, :hq // hkv]).all()
    assert torch.isfinite(o[:2, hq // hkv:]).all() and torch.isfinite(o[2:]).all()


def test_far_offsets():
    """Pages whose element offsets pass 2^31."""
    d, hkv, page, dtype = 128, 2, 16, torch.bfloat16
    rng = np.random.default_rng(3)
    ctx, new = [40, 30], [2, 1]
    small = R.make_cache(rng, [a + b for a, b in zip(ctx, new)], hkv, d, page, dtype)
    stride = (1 << 29) + 64
    big = stride * (small.n_pages - 1) + page * hkv * d
    assert big > 1 << 31
    q = torch.randn((3, 8, d), generator=torch.Generator().manual_seed(1)).to(dtype)
    a = Attn(small, q, ctx, new, None, dtype, d ** -0.5)
    want = a.out()
    pools = []
    for src in (a.k, a.v):
        t = torch.empty(big, dtype=dtype, device="cuda")
        for p in range(small.n_pages):
            t[p * stride:p * stride + page * hkv * d] = src[p * page * hkv * d:(p + 1) * page * hkv * d]
        pools.append(t)
    a.k, a.v = pools
    a.dm.page_stride = stride
    a.o.fill_(float("nan"))
    assert torch.equal(a.out(), want)


def test_repeats_bit_for_bit_and_on_another_stream():
    dtype, d = torch.bfloat16, 256
    ctx = [900, 10, 300, 2500]
    cache, q, _ = case(12, dtype, d, 16, 2, 16, "token", ctx, [1] * 4, False)
    a = Attn(cache, q, ctx, [1] * 4, None, dtype, d ** -0.5)
    want = a.out()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        a.o.fill_(float("nan"))
        torch.cuda.synchronize()
        a(stream=st)
        torch.cuda.synchronize()
        assert torch.equal(a.o.cpu(), want)


@pytest.mark.parametrize("what,code", [("page", G.GDN_DEV_BAD_PAGE), ("len", G.GDN_DEV_BAD_LEN), ("neg", G.GDN_DEV_BAD_LEN),
                                       ("off", G.GDN_DEV_BAD_NODE_OFF), ("many", G.GDN_DEV_BAD_NODE_OFF),
                                       ("parent", G.GDN_DEV_BAD_PARENT)])
def test_attention_device_errors(what, code):
    dtype, d = torch.bfloat16, 256
    ctx, new = [100, 50], [8, 8]
    cache, q, parents = case(13, dtype, d, 16, 2, 16, "token", ctx, new, True)
    a = Attn(cache, q, ctx, new, parents, dtype, d ** -0.5, max_tokens=7 if what == "many" else None)
    if what == "page":
        a.table[1, 2] = cache.n_pages
    elif what == "len":
        a.ctx[1] = cache.table.shape[1] * 16 - 3
    elif what == "neg":
        a.ctx[0] = -1
    elif what == "off":
        a.off[1] = 17
    elif what == "parent":
        a.par[10] = 5
    a()
    torch.cuda.synchronize()
    assert int(a.status) == code


# ---- rope and append ---------------------------------------------------------------------------------------------------------


def run_rope(cache, q, k, v, ctx, new, pos, inv_freq, axis, rot, inter, qw, kw, eps, dtype, in_place=False, pad=0):
    N, hq, d = q.shape
    dm = gdims(cache, new, hq, dtype)
    dev = [cache.k.cuda(), cache.v.cuda()]
    rows = []
    for x in (q, k, v):
        b = torch.full((N, x.shape[1] * d + pad), float("nan"), dtype=dtype)
        b[:, :x.shape[1] * d] = x.reshape(N, -1)
        rows.append(b.cuda())
    qo = rows[0] if in_place else torch.full((N, hq * d), float("nan"), dtype=dtype, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    f = torch.tensor(inv_freq, dtype=torch.float64, device="cuda") if rot else None
    G.gdn_rope_append(dm, rows[0], rows[0].stride(0), rows[1], rows[1].stride(0), rows[2], rows[2].stride(0),
                      None if qw is None else qw.cuda(), None if kw is None else kw.cuda(), eps,
                      i32(pos), pos.shape[1], f, None if axis is None else i32(axis), rot, int(inter), i32(offsets(new)),
                      i32(ctx), i32(cache.table), qo, qo.stride(0), dev[0], dev[1], status)
    torch.cuda.synchronize()
    assert int(status) == 0
    return qo.cpu()[:, :hq * d].reshape(N, hq, d), dev[0].cpu(), dev[1].cpu()


@pytest.mark.parametrize("d,hq,hkv,rot,inter,axes,norm,name,layout", [
    (256, 16, 2, 64, False, 3, True, "bf16", "token"), (256, 5, 1, 256, False, 1, False, "fp16", "head"),
    (128, 6, 3, 128, True, 3, True, "bf16", "padded"), (128, 7, 7, 16, False, 2, False, "bf16", "token"),
    (64, 9, 3, 64, False, 4, True, "fp16", "token"), (64, 4, 4, 32, True, 1, False, "bf16", "head"),
    (256, 3, 3, 0, False, 1, True, "bf16", "token")])
def test_rope_append(d, hq, hkv, rot, inter, axes, norm, name, layout):
    dtype = R.DTYPES[name]
    rng = np.random.default_rng(d + hq)
    ctx, new = [13, 0, 31], [5, 0, 18]
    cache = R.make_cache(rng, [a + b for a, b in zip(ctx, new)], hkv, d, 16, dtype, layout, garbage=77.0)
    g = torch.Generator().manual_seed(d)
    N = sum(new)
    q, k, v = (torch.randn((N, h, d), generator=g).to(dtype) for h in (hq, hkv, hkv))
    v[0, 0, :4] = torch.tensor([float("nan"), float("inf"), -0.0, 1e-7]).to(dtype)
    pos = rng.integers(-50, 2_000_000, (N, axes))
    pos[0] = 0
    pos[1] = 2 ** 31 - 1
    inv_freq = [1e6 ** (-i / max(rot // 2, 1)) for i in range(rot // 2)]
    axis = [int(x) for x in rng.integers(0, axes, rot // 2)]
    qw = (1 + 0.2 * torch.randn(d, generator=g)) if norm else None
    kw = (1 + 0.2 * torch.randn(d, generator=g)) if norm else None
    eps = 1e-6
    before = cache.k.clone(), cache.v.clone()
    qo, kp, vp = run_rope(cache, q, k, v, ctx, new, pos, inv_freq, axis, rot, inter, qw, kw, eps, dtype, pad=8)
    h = R.half_step(dtype)
    tiny = torch.finfo(dtype).smallest_normal * h          # below the normal range the step is fixed
    zq, mq = R.rope(q.double(), pos, inv_freq, axis, rot, inter, None if qw is None else qw.double(), eps)
    zk, mk = R.rope(k.double(), pos, inv_freq, axis, rot, inter, None if kw is None else kw.double(), eps)
    # 2^31 turns of a double's 2^-53 are 2^-22 of a turn: the farthest position gets that much more
    far = np.abs(pos).max(1) > 2 ** 24
    slack = torch.tensor(np.where(far, 2.0 ** -18, 2.0 ** -19)).view(-1, 1, 1)
    assert bool(((qo.double() - zq).abs() <= h * zq.abs() + slack * mq + tiny).all())
    exp_k, exp_v, n = before[0].double(), before[1].clone(), 0
    tol = torch.zeros_like(exp_k)
    for s, c in enumerate(new):
        for i in range(c):
            at = cache.index(s, ctx[s] + i)
            exp_k[at] = zk[n]
            tol[at] = h * zk[n].abs() + slack[n] * mk[n] + tiny
            exp_v[at] = v[n]
            n += 1
    assert bool(((kp.double() - exp_k).abs() <= tol).all())             # untouched places exactly
    assert torch.equal(vp.view(torch.int16), exp_v.view(torch.int16))   # values bit for bit, NaN among them
    if norm:                                                            # in place gives the same
        qi, _, _ = run_rope(cache, q, k, v, ctx, new, pos, inv_freq, axis, rot, inter, qw, kw, eps, dtype, in_place=True, pad=8)
        assert torch.equal(qi, qo)


def test_rope_many_tokens_and_sequences():
    """More tokens than warps that fill the GPU (one warp a token), 700 sequences."""
    d, hq, hkv, dtype = 64, 4, 2, torch.bfloat16
    rng = np.random.default_rng(2)
    new = [int(x) for x in rng.integers(0, 14, 700)]
    ctx = [int(x) for x in rng.integers(0, 20, 700)]
    cache = R.make_cache(rng, [a + b for a, b in zip(ctx, new)], hkv, d, 8, dtype, garbage=1.0)
    N = sum(new)
    assert N > 152 * 24
    g = torch.Generator().manual_seed(4)
    q, k, v = (torch.randn((N, h, d), generator=g).to(dtype) for h in (hq, hkv, hkv))
    pos = rng.integers(0, 100, (N, 1))
    inv_freq = [1e4 ** (-i / 32) for i in range(32)]
    qo, kp, vp = run_rope(cache, q, k, v, ctx, new, pos, inv_freq, None, 64, False, None, None, 0.0, dtype)
    zq, mq = R.rope(q.double(), pos, inv_freq, [0] * 32, 64, False)
    assert bool(((qo.double() - zq).abs() <= R.half_step(dtype) * zq.abs() + 2.0 ** -19 * mq).all())
    off = offsets(new)
    for s in range(0, 700, 37):
        for i in range(new[s]):
            assert torch.equal(vp[cache.index(s, ctx[s] + i)], v[off[s] + i])


def test_rope_device_errors():
    d, dtype = 64, torch.bfloat16
    rng = np.random.default_rng(2)
    ctx, new = [10, 20], [4, 4]
    cache = R.make_cache(rng, [14, 24], 2, d, 8, dtype)
    base = dict(off=offsets(new), ctx=ctx, table=cache.table, axis=[0] * 8)
    for what, code in (("page", G.GDN_DEV_BAD_PAGE), ("len", G.GDN_DEV_BAD_LEN), ("neg", G.GDN_DEV_BAD_LEN),
                       ("off", G.GDN_DEV_BAD_NODE_OFF), ("axis", G.GDN_DEV_BAD_AXIS)):
        a = {x: np.array(y) for x, y in base.items()}
        if what == "page":
            a["table"][0, 1] = -1
        elif what == "len":
            a["ctx"][1] = cache.table.shape[1] * 8 - 2
        elif what == "neg":
            a["ctx"][1] = -5
        elif what == "off":
            a["off"][1] = 9
        else:
            a["axis"][3] = 1
        q = torch.zeros(8, 128, dtype=dtype, device="cuda")
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        G.gdn_rope_append(gdims(cache, new, 2, dtype), q, 128, torch.zeros_like(q), 128, torch.zeros_like(q), 128, None, None,
                          0.0, i32([[1]] * 8), 1, torch.ones(8, dtype=torch.float64, device="cuda"), i32(a["axis"]), 16, 0,
                          i32(a["off"]), i32(a["ctx"]), i32(a["table"]), torch.empty_like(q), 128, cache.k.cuda(),
                          cache.v.cuda(), status)
        torch.cuda.synchronize()
        assert int(status) == code, what


# ---- commit in the cache -----------------------------------------------------------------------------------------------------


def run_move(cache, layers, stride, kbuf, vbuf, ctx, new, parents, acc, dtype, status0=0, **over):
    dm = gdims(cache, new, cache.h_kv, dtype)
    k, v = kbuf.cuda(), vbuf.cuda()
    nl = torch.full((max(len(new), 1),), -7, dtype=torch.int32, device="cuda")
    status = torch.full((1,), status0, dtype=torch.int32, device="cuda")
    par = i32([x for p in parents for x in p])
    G.gdn_kv_commit(dm, layers, stride, i32(acc), par, i32(over.get("off", offsets(new))), i32(ctx),
                    i32(over.get("table", cache.table)), k, v, nl, status)
    torch.cuda.synchronize()
    return k.cpu(), v.cpu(), nl.cpu().tolist(), int(status)


@pytest.mark.parametrize("d,hkv,page,layout,kind", [
    (256, 2, 16, "token", "tree"), (128, 8, 8, "head", "tree"), (64, 3, 32, "padded", "tree"), (64, 1, 8, "token", "chain"),
    (256, 5, 64, "token", "star")])
def test_move(d, hkv, page, layout, kind):
    dtype = torch.bfloat16
    rng = np.random.default_rng(d + hkv)
    ctx, new = [5, 0, 40, 9, 17], [16, 0, 64, 1, 33]
    cache = R.make_cache(rng, [a + b for a, b in zip(ctx, new)], hkv, d, page, dtype, layout, garbage=3.0)
    parents = [R.random_tree(rng, n) if kind == "tree" and n else [i - 1 for i in range(n)] if kind == "chain"
               else [-1] + [0] * (n - 1) if n else [] for n in new]
    acc = [11, -1, 63, -1, 30]
    layers, size = 3, cache.k.numel()
    stride = (size + 15) // 8 * 8
    g = torch.Generator().manual_seed(1)
    k, v = (torch.randn(stride * (layers - 1) + size, generator=g).to(dtype) for _ in range(2))
    ek, ev = k.clone(), v.clone()
    lens = list(ctx)
    for s, n in enumerate(new):
        if acc[s] < 0:
            continue
        path = R.path_of(parents[s], acc[s])
        lens[s] += len(path)
        for buf, src in ((ek, k), (ev, v)):
            for layer in range(layers):
                for j, x in enumerate(path):
                    buf[layer * stride + cache.index(s, ctx[s] + j)] = src[layer * stride + cache.index(s, ctx[s] + x)]
    gk, gv, nl, status = run_move(cache, layers, stride, k, v, ctx, new, parents, acc, dtype)
    assert status == 0 and nl == lens
    assert torch.equal(gk, ek) and torch.equal(gv, ev)


@pytest.mark.parametrize("what,code", [("accepted", G.GDN_DEV_BAD_ACCEPTED), ("parent", G.GDN_DEV_BAD_PARENT),
                                       ("page", G.GDN_DEV_BAD_PAGE), ("len", G.GDN_DEV_BAD_LEN),
                                       ("off", G.GDN_DEV_BAD_NODE_OFF), ("status", 3)])
def test_move_is_a_transaction(what, code):
    """A fault in one sequence, or an earlier one, and nothing is written."""
    d, dtype = 64, torch.bfloat16
    rng = np.random.default_rng(6)
    ctx, new = [5, 12], [8, 8]
    cache = R.make_cache(rng, [13, 20], 2, d, 8, dtype, garbage=2.0)
    parents, acc, over = [[-1, 0, 0, 1, 1, 2, 2, 3]] * 2, [7, 6], {}
    if what == "accepted":
        acc = [7, 8]
    elif what == "parent":
        parents = [parents[0], [-1, 0, 0, 1, 1, 2, 6, 3]]
    elif what == "page":
        over["table"] = cache.table.copy()
        over["table"][1, 2] = 99
    elif what == "len":
        over["ctx"] = [5, cache.table.shape[1] * 8 - 7]
    elif what == "off":
        over["off"] = [0, 8, 15]
    k, v, nl, status = run_move(cache, 1, 0, cache.k, cache.v, over.pop("ctx", ctx), new, parents, acc, dtype,
                                status0=3 if what == "status" else 0, **over)
    assert status == code and nl == [-7, -7]
    assert torch.equal(k, cache.k) and torch.equal(v, cache.v)
