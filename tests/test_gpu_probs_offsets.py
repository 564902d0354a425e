"""Offsets of sequences that are out of order where no row comes to them: reported all the same."""
import pytest
import torch

import gated_deltanet_speculative_gdn_gb300 as G

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # collected on CPU machines, never run there
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from test_gpu_probs import Probs, i32  # noqa: E402

BAD = [
    [0, 8, 12, 8],      # past the last row, and back
    [0, 8, 8, 12],      # the last one past the last row
    [0, 5, 3, 8],       # a sequence that ends before it begins
    [0, -2, 1, 8],
    [0, 3, 9, 8],
]


@pytest.mark.parametrize("off", BAD)
def test_few_rows(off):
    c = Probs(1, "bf16", 500, [8, 0, 0], False)
    c.rep = c.freq = c.pres = c.temp = None           # (without what would be read by sequence)
    c.call(off=i32(off))
    assert int(c.status) == G.GDN_DEV_BAD_NODE_OFF
    c.call()
    assert int(c.status) == 0
