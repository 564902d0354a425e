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

from attn_long import Call  # noqa: E402


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
