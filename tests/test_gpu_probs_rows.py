"""Rows that the same CTAs of gdn_logits_probs work through one after the other: nothing of one row reaches the next."""
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # collected on CPU machines, never run there
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import gated_deltanet_speculative_gdn_gb300 as G  # noqa: E402
from test_gpu_probs import Probs, i32  # noqa: E402


@pytest.mark.parametrize("name,V,new", [("bf16", 65536, [16] * 20), ("fp32", 131072, [8] * 12), ("fp16", 16384, [3, 40] * 16)])
def test_rows_that_differ(name, V, new):
    """Logits of another place and size in every row, paths, biases and masks that come and go; the same bits every time."""
    c = Probs(150, name, V, new, True)
    n = torch.arange(c.N)
    c.logits[:, :V] = (c.logits[:, :V].float() + 20.0 * (n % 5).view(-1, 1)).to(c.dtype)
    for k in range(6):
        c.logits[n, (n * 1999 + 8 * k) % V] = 100.0
    c.biases([0 if s % 3 == 0 else 30 for s in range(c.S)]).masks([k if k % 2 else -1 for k in range(c.N)], share=0.3)
    c.temp[1::4] = 0
    c.check()
    first = c.call()
    for _ in range(10):
        assert torch.equal(c.call(), first) and int(c.status) == 0


def test_offsets_out_of_order():
    """As in test_gpu_probs_offsets.py, for 320 rows."""
    good = list(range(0, 321, 64))
    c = Probs(1, "bf16", 16384, [64] * 5, False)
    c.rep = c.freq = c.pres = c.temp = None
    for off, code in ((good, 0), (good + [321], G.GDN_DEV_BAD_NODE_OFF), (good + [300, 320], G.GDN_DEV_BAD_NODE_OFF),
                      (good + [-1, 320], G.GDN_DEV_BAD_NODE_OFF), (good[:-1] + [384, 320], G.GDN_DEV_BAD_NODE_OFF), (good, 0)):
        c.S = len(off) - 1
        c.call(off=i32(off))
        assert int(c.status) == code, off
