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
