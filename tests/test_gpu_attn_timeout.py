"""The attention kernel when a wait runs out: one role of the first CTA gives up (a test
hook makes it wait for what never comes), the others wait out their limits, drain their
copies and products and leave; the call reports it and the context goes on."""
import pytest
import torch

import gated_deltanet_speculative_gdn_gb300 as G

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # collected on CPU machines, never run there
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from attn_long import Call  # noqa: E402


@pytest.mark.parametrize("name,d,hq,hkv", [("bf16", 256, 16, 2), ("fp16", 128, 8, 2), ("bf16", 64, 4, 4)])
@pytest.mark.parametrize("role", range(5))
@pytest.mark.parametrize("ctx", [[5] * 240, [5] + [900] * 120])
def test_wait_that_runs_out_reports_timeout_and_the_context_survives(name, d, hq, hkv, role, ctx):
    """With a share that the copies' warp can request whole before anyone takes it, and with one that is longer
    than the ring; the first items are trees, so that values are cleaned."""
    if len(set(ctx)) == 1:
        ctx = ctx[:240 // hkv]   # 11 units an item, 17 a CTA: the first CTA has one tile and the next item's front
    a = Call(3, name, d, hq, hkv, 16, ctx, [7] * len(ctx), tree=True)
    want = a.out()
    G.gdn_test_stall_next_attention(20_000_000, role)
    a()
    torch.cuda.synchronize()
    assert int(a.status) == G.GDN_DEV_TIMEOUT, G.gdn_status_str(int(a.status))
    a.status.zero_()
    assert torch.equal(a.out(), want)
