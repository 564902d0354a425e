"""Values that are NaN at positions of the 4-bit cache whose weights underflow."""
import numpy as np
import pytest
import torch

import kv4_ref as Q

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # collected on CPU machines, never run there
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from test_gpu_attn_kvq import Attn4  # noqa: E402


@pytest.mark.parametrize("S", [1, 400])                       # over many CTAs, and several sequences in one
@pytest.mark.parametrize("d,new", [(256, 1), (128, 1), (128, 4), (64, 3), (256, 20), (64, 40)])
def test_nan_values_of_positions_that_count_for_nothing(d, new, S):
    """A value that is NaN is NaN times whatever weight its position has, one that underflows too: every fourth tile of
    64 positions has scores hundreds below the others', and a NaN.  (The sequences have the same pages.)"""
    dtype, ctx = torch.float16, 500
    cache = Q.make_cache4(np.random.default_rng(34), [ctx + new], 2, d, 16)
    for x in range(ctx + new):
        cache.put(cache.k, 0, x, torch.full((2, d), -6.0 if x // 64 % 4 == 0 else 6.0, dtype=torch.float64), 1.0)
    cache.v[cache.scales_at(0, 3)[1, 2]] = 0x7f               # head 1, columns 32 .. 47
    cache.table = np.repeat(cache.table, S, axis=0)
    q = torch.full((S * new, 8, d), 4.0, dtype=dtype)
    a = Attn4(cache, q, [ctx] * S, [new] * S, None, dtype, d ** -0.5)
    o = a.out()
    want = torch.zeros(S * new, 8, d, dtype=torch.bool)
    want[:, 4:, 32:48] = True
    assert int(a.status) == 0 and torch.equal(torch.isnan(o), want)
