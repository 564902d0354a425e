"""Attention over the 4-bit cache where a factor leaves the range of its type: scales and units at the ends of what is
allowed, and rows of zeros.

Tolerances: those of test_gpu_attn_kvq.py."""
import numpy as np
import pytest
import torch

import attn_ref as R
import gated_deltanet_speculative_gdn_gb300 as G
import kv4_ref as Q

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # collected on CPU machines, never run there
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from test_gpu_attn_kvq import Attn4, check, sum_of_values  # noqa: E402

CTX = [300, 5]
# new tokens of a group of four: few rows (one and two blocks of eight), and the long chunks' kernel
FORMS = [(256, [1, 2]), (128, [4, 1]), (64, [3, 1]), (256, [20, 3]), (128, [40, 1]), (64, [17, 2])]


def cache_of(seed, d, new, units, std=1.0):
    rng = np.random.default_rng(seed)
    return Q.make_cache4(rng, [a + b for a, b in zip(CTX, new)], 2, d, 16, "dense", units, std=std)


def compare(cache, q, new, dtype, scale, d):
    ref, A, big = R.attention(q.double(), cache, CTX, new, None, scale)
    a = Attn4(cache, q, CTX, new, None, dtype, scale)
    o = a.out()
    assert int(a.status) == 0
    check(o, ref, A, sum_of_values(cache, CTX, new, q.shape[1]), big, dtype, d)


@pytest.mark.parametrize("d,new", FORMS)
@pytest.mark.parametrize("scale", [2.0 ** -27, 1e-38, 1e-45])
@pytest.mark.parametrize("name", ["bf16", "fp16"])
def test_small_scales(name, scale, d, new):
    """A factor that underflows: all positions that a row sees weigh alike, the masked ones nothing."""
    dtype = R.DTYPES[name]
    cache = cache_of(31, d, new, (2.0 ** -24, 1.0))
    g = torch.Generator().manual_seed(d)
    q = torch.randn((sum(new), 8, d), generator=g).to(dtype)
    q[0] = 0
    compare(cache, q, new, dtype, scale, d)


@pytest.mark.parametrize("d,new", FORMS)
def test_large_queries_bring_a_small_scale_back(d, new):
    """scale * k_unit is below fp32's range, times the queries it is not: keys of up to 2^9 units, queries of 2^122 and
    a scale of 2^-107 make scores of a few units."""
    cache = cache_of(32, d, new, (2.0 ** -24, 1.0), std=100.0)
    g = torch.Generator().manual_seed(d)
    q = (torch.randn((sum(new), 8, d), generator=g) * 2.0 ** 122).to(torch.bfloat16)
    scale = 2.0 ** -107
    ref, A, big = R.attention(q.double(), cache, CTX, new, None, scale)
    flat, _, _ = R.attention(torch.zeros_like(q).double(), cache, CTX, new, None, scale)
    assert float((ref - flat).abs().max()) > 0.01          # the scores say something
    a = Attn4(cache, q, CTX, new, None, torch.bfloat16, scale)
    o = a.out()
    assert int(a.status) == 0
    check(o, ref, A, sum_of_values(cache, CTX, new, 8), big, torch.bfloat16, d)


@pytest.mark.parametrize("d,new", FORMS)
def test_large_scales(d, new):
    """A factor that overflows, of scores that are 0: keys of zeros."""
    cache = cache_of(33, d, new, (1.0, 1.0))
    for s, (c, n) in enumerate(zip(CTX, new)):
        for x in range(c + n):
            cache.put(cache.k, s, x, torch.zeros(2, d, dtype=torch.float64), 1.0)
    g = torch.Generator().manual_seed(d)
    q = (torch.randn((sum(new), 8, d), generator=g) * 2.0 ** 120).to(torch.bfloat16)
    compare(cache, q, new, torch.bfloat16, 2.0 ** 30, d)


@pytest.mark.parametrize("new", [[1, 1], [24, 3]])
def test_far_pages(new):
    """Pages 2^30 bytes apart, read beyond 2^32."""
    d, hkv, page, stride, n_pages, dtype = 64, 2, 16, 1 << 30, 7, torch.bfloat16
    ctx = [40, 3]
    near = Q.make_cache4(np.random.default_rng(35), [a + b for a, b in zip(ctx, new)], hkv, d, page, extra=0)
    block = G.gdn_kvq_block_bytes(G.AttnDims.make_kvq(1, 1, 1, 8, hkv, d, G.GDN_BF16, 1, page, 1))
    q = torch.randn((sum(new), 8, d), generator=torch.Generator().manual_seed(5)).to(dtype)
    ref, A, big = R.attention(q.double(), near, ctx, new, None, d ** -0.5)
    assert near.n_pages <= n_pages
    a = Attn4(near, q, ctx, new, None, dtype, d ** -0.5)
    far = [torch.empty((n_pages - 1) * stride + hkv * block, dtype=torch.uint8, device="cuda") for _ in range(2)]
    for to, buf in zip(far, (near.k, near.v)):
        for p in range(near.n_pages):
            at = (n_pages - 1 - p) * stride                   # the first pages last
            to[at:at + hkv * block] = buf[p * hkv * block:(p + 1) * hkv * block].cuda()
    a.k, a.v = far
    a.table = torch.where(a.table < near.n_pages, n_pages - 1 - a.table, a.table)
    a.dm = G.AttnDims.make_kvq(2, sum(new), max(new), 8, hkv, d, G.GDN_BF16, n_pages, page, near.table.shape[1], stride, block)
    o = a.out()
    assert int(a.status) == 0
    check(o, ref, A, sum_of_values(near, ctx, new, 8), big, dtype, d)
