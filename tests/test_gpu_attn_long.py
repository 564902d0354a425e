"""Paged attention where a CTA works through many tiles and items: what the small
cases of the attention tests do not reach.  Each test states what of the schedule it
reaches, from a copy of the schedule, so that it cannot shrink unseen."""
import numpy as np
import pytest
import torch

import attn_ref as R

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # collected on CPU machines, never run there
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from attn_long import FRONT, TILE, Call, item_tiles  # noqa: E402


@pytest.mark.parametrize("name,d,hq,hkv,page,tree", [
    ("bf16", 256, 16, 2, 16, True), ("fp16", 256, 6, 1, 64, False), ("fp16", 128, 10, 2, 32, True),
    ("bf16", 128, 8, 2, 16, False), ("bf16", 64, 5, 1, 8, True), ("fp16", 64, 8, 8, 64, False)])
def test_rows_of_a_warp_go_other_ways(name, d, hq, hkv, page, tree):
    """Row tiles that end inside a warp, and values that are not finite which some rows of a warp see and others
    do not, at the ends of many items of a CTA: the rows that do not see them keep their results bit for bit."""
    new = [int(x) for x in np.random.default_rng(d).integers(3, 61, 150)]
    ctx = [int(x) for x in np.random.default_rng(d + 1).integers(0, 1500, 150)]
    a = Call(1, name, d, hq, hkv, page, ctx, new, tree)
    r = a.reached()
    assert r["segments"] >= 2 and r["tiles"] >= 8, r
    clean = a.out()
    a.check(clean, range(0, 150, 17))
    free = torch.ones(a.N, dtype=torch.bool, device="cuda")
    where = {}
    for s in range(0, 150, 3):
        i = new[s] // 2
        where[s] = i
        row = int(a.rows(s)[ctx[s] + i])
        a.v[row, :, 3] = [float("nan"), float("inf"), float("-inf")][(s // 3) % 3]
        free[int(a.off[s]):int(a.off[s + 1])] = ~a.seen(s)[:, ctx[s] + i]
    dirty = a.out()
    assert torch.equal(dirty[free], clean[free])
    assert not torch.isfinite(dirty[~free][..., 3]).any()
    other = [c for c in range(d) if c != 3]
    assert torch.equal(dirty[..., other], clean[..., other])


@pytest.mark.parametrize("d", [256, 128, 64])
@pytest.mark.parametrize("name", ["fp16", "bf16"])
@pytest.mark.parametrize("gap", [10.0, 16.0, 18.0])
def test_weights_far_below_the_largest(name, d, gap):
    """The first key of a long context stands `gap` (nats) above 16,384 others, as a sequence's first token may, and
    its value is a hundredth of theirs: the small weights carry a share of the result that no type may lose.  One
    sequence a CTA, all over the same pages, so that one running maximum holds for all of them."""
    S = torch.cuda.get_device_properties(0).multi_processor_count
    pages = np.random.default_rng(0).permutation(259)[:257]
    a = Call(5, name, d, 8, 1, 64, [16384] * S, [1] * S, pages_of=[pages] * S, n_pages=259)
    assert a.reached()["longest"] >= 257
    g = torch.Generator(device="cuda").manual_seed(6)
    a.q.zero_()
    a.q[..., 0] = gap * d ** 0.5
    a.q[..., 1:8] = (torch.randn((a.N, 8, 7), generator=g, device="cuda") * 0.2 * d ** 0.5).to(a.dtype)
    rows = a.rows(0)
    a.k[rows] = 0.0
    a.k[rows, :, 1:8] = torch.randn((len(rows), 1, 7), generator=g, device="cuda").to(a.dtype)
    a.k[rows[0]] = 0.0
    a.k[rows[0], :, 0] = 1.0
    a.v[rows] = (0.5 + torch.rand((len(rows), 1, d), generator=g, device="cuda")).to(a.dtype)
    a.v[rows[0]] = 0.01
    a.check(a.out(), terms=8)


@pytest.mark.parametrize("name,d,hq,hkv,page,tree", [
    ("bf16", 256, 16, 2, 32, True), ("fp16", 256, 16, 2, 64, False), ("fp16", 128, 8, 2, 16, False),
    ("bf16", 64, 8, 4, 8, True)])
def test_sequences_that_share_the_pages_of_a_prefix(name, d, hq, hkv, page, tree):
    """48 sequences over one prefix of 4,096 positions, each with up to 150 of its own."""
    S, pre, rng = 48, 4096, np.random.default_rng(d)
    own, new = rng.integers(0, 150, S), rng.integers(1, 20, S)
    need = [-(-(int(a) + int(b)) // page) for a, b in zip(own, new)]
    perm, at, pages = rng.permutation(pre // page + sum(need)), pre // page, []
    for k in need:
        pages.append(np.concatenate([perm[:pre // page], perm[at:at + k]]))
        at += k
    a = Call(9, name, d, hq, hkv, page, pre + own, new, tree, pages_of=pages, n_pages=len(perm))
    r = a.reached()
    assert r["tiles"] >= 24 and r["both"] >= 1, r
    o = a.out()
    a.check(o)
    assert torch.equal(a.out(), o)


def lengths(kind, seed):
    """(ctx, new) of prompts' chunks of several row tiles, of trees over long contexts, or of few long sequences."""
    rng = np.random.default_rng(seed)
    if kind == "chunks":
        return rng.integers(0, 3000, 9), rng.integers(130, 420, 9)
    if kind == "trees":
        return rng.integers(500, 6000, 40), rng.integers(0, 41, 40)
    return np.array([70001, 5, 33333, 0]), np.array([3, 1, 2, 17])


LONG = [(name, d, hq, hkv, page, kind)
        for d, heads in ((256, ((16, 2), (6, 2))), (128, ((10, 2), (16, 4))), (64, ((16, 8), (14, 2))))
        for (hq, hkv), name, pages in zip(heads, ("bf16", "fp16"), ((8, 32, 64), (64, 16, 8)))
        for page, kind in zip(pages, ("chunks", "trees", "long"))]


@pytest.mark.parametrize("name,d,hq,hkv,page,kind", LONG)
def test_long_work(name, d, hq, hkv, page, kind):
    """More tiles a CTA than its ring holds (6, 12 or 24 stages of one tile's keys or values), several items a CTA
    with an end of one and a beginning of another, segments of more pages than the 64 table entries that are loaded
    ahead.  Every output against 64 bits, and the same bits again."""
    ctx, new = lengths(kind, d)
    a = Call(20, name, d, hq, hkv, page, ctx, new, tree=kind == "trees")
    r = a.reached()
    stages = 196608 // (TILE * d * 2)
    assert r["total"] >= 16 * 152 and r["tiles"] * 2 > min(stages, 20) and r["both"] > 0, r
    if kind != "long":
        assert r["segments"] >= 2, r
    elif page == 8:
        assert r["longest"] * TILE // page > 64, r
    o = a.out()
    a.check(o)
    for _ in range(3):
        assert torch.equal(a.out(), o)


@pytest.mark.parametrize("d", [256, 128, 64])
@pytest.mark.parametrize("name", ["bf16", "fp16"])
@pytest.mark.parametrize("std", [1e-3, 8.0])
def test_long_flat_and_peaked(name, d, std):
    """Nearly equal scores, and scores that make a few positions take all, along whole contexts of one CTA."""
    a = Call(21, name, d, 16, 2, 64, [4000] * 80, [5] * 80, tree=True, q_std=std)
    assert a.reached()["longest"] >= 60
    a.check(a.out())


@pytest.mark.parametrize("d", [256, 128, 64])
@pytest.mark.parametrize("name", ["bf16", "fp16"])
@pytest.mark.parametrize("step,moves", [(2e-5, False), (1e-3, True), (2e-2, True), (-2e-2, False)])
def test_scores_that_rise_along_the_context(name, d, step, moves):
    """Keys that grow (or shrink) along the context, so that the largest score rises from tile to tile by less than
    what moves a row's reference, by as much in some tiles, by more in every one, or falls.  All sequences over the
    same pages, an item or more a CTA."""
    S = 2 * torch.cuda.get_device_properties(0).multi_processor_count
    pages = np.random.default_rng(1).permutation(66)[:65]
    a = Call(22, name, d, 4, 1, 64, [4096] * S, [2] * S, pages_of=[pages] * S, n_pages=66)
    assert a.reached()["longest"] >= 60
    a.q.abs_()
    rows = a.rows(0)
    x = torch.arange(len(rows), device="cuda") if step > 0 else torch.arange(len(rows), 0, -1, device="cuda")
    a.k[rows] = (a.k[rows].float().abs() * abs(step) * x[:, None, None]).to(a.dtype)
    # how far the largest score of a tile lies above that of the tiles before it, in bits, over the sequences' rows
    top = (a.q.double().view(-1, d) @ a.k[rows[:4096], 0].double().T * a.scale * 1.4426950408889634).view(-1, 64, TILE).amax(-1)
    rise = top[:, 1:].cummax(1).values - top[:, :1]
    if step < 0:
        assert bool((top[:, 32:].amax(1) < top[:, :32].amax(1) - 16.5).all())
    else:
        assert bool((rise.amax(1) > 16.5).all()) if moves else bool((rise < 7.5).all())
    a.check(a.out(), range(0, S, 7))


def test_nan_keys_in_long_contexts_reach_the_rows_that_see_them_alone():
    for name, d in (("bf16", 256), ("fp16", 128), ("bf16", 64)):
        a = Call(23, name, d, 8, 2, 16, [3000] * 60, [2] * 60)
        assert a.reached()["segments"] >= 1 and a.reached()["tiles"] >= 30
        want = a.out()
        for s in range(0, 60, 4):
            a.k[a.rows(s)[100 + 40 * s:101 + 41 * s], 1] = float("nan")
        o = a.out().view(60, 2, 2, 4, d)
        hit = torch.zeros((60, 2), dtype=torch.bool, device="cuda")
        hit[::4, 1] = True
        assert torch.isnan(o.transpose(1, 2)[hit]).all()
        assert torch.equal(o.transpose(1, 2)[~hit], want.view(60, 2, 2, 4, d).transpose(1, 2)[~hit])


@pytest.mark.parametrize("name,d,hq,hkv,S", [("bf16", 256, 8, 1, 1000), ("fp16", 128, 4, 2, 777), ("bf16", 64, 8, 2, 3000)])
def test_more_sequences_than_threads(name, d, hq, hkv, S):
    """Several sequences to a thread of the schedule, empty ones among them."""
    rng = np.random.default_rng(S)
    ctx, new = rng.integers(0, 400, S), rng.integers(0, 12, S) * (rng.random(S) < 0.7)
    table = rng.integers(0, 500, (S, 52))
    a = Call(24, name, d, hq, hkv, 8, ctx, new, tree=True, table=table, n_pages=500)
    o = a.out()
    a.check(o)
    assert torch.equal(a.out(), o)


def test_more_units_than_32_bits_of_products():
    """60,000 short sequences of 16 heads: 157 sequences to a thread, and shares that are cut in 64 bits."""
    S = 60000
    rng = np.random.default_rng(2)
    ctx = rng.integers(0, 63, S)
    a = Call(25, "fp16", 64, 16, 16, 16, ctx, [1] * S, table=rng.integers(0, 4096, (S, 4)), n_pages=4096)
    tiles = item_tiles(ctx, [1] * S, 16, 1)
    assert int((tiles + FRONT).sum()) >= 1 << 23
    o = a.out()
    assert torch.isfinite(o).all()
    a.check(o, range(0, S, 199))


def test_contexts_of_16_million_positions():
    """Four sequences of 2^24 positions and eight heads, 2^23 units and shares that begin far into an item.  All
    scores are equal and the values of the r-th of 64 regions of a context are 1 in column r and 0 elsewhere, so every
    output is exactly a 64th: 16 of a region's 4,096 tiles lost or taken twice would show."""
    S, L = 4, 1 << 24
    table = np.tile(np.arange(L // 64) // (L // 64 // 64), (S, 1))
    a = Call(26, "bf16", 64, 8, 8, 64, [L - 1] * S, [1] * S, table=table, n_pages=64)
    assert int((item_tiles(a.ctx, a.new, 8, 1) + FRONT).sum()) >= 1 << 23
    a.q.zero_()
    a.v.zero_()
    for r in range(64):
        a.v[64 * r:64 * (r + 1), :, r] = 1.0
    o = a.out().double()
    assert float((o * 64 - 1).abs().max()) <= R.half_step(torch.bfloat16)
