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
