"""The 4-bit cache's attention and the probabilities on two streams at once, each with buffers of its own: the bits of
calls one after the other."""
import pytest
import torch

import gated_deltanet_speculative_gdn_gb300 as G

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # collected on CPU machines, never run there
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from test_gpu_attn_kvq import Attn4, case  # noqa: E402
from test_gpu_probs import Probs  # noqa: E402


class ProbsCall:
    """A call whose tensors are on the GPU already."""

    def __init__(self, c):
        self.c = c
        self.want = c.call()
        self.out = torch.full_like(self.want, 7.0)                # (as there: what is past the vocabulary stays)
        self.dm = G.GdnDims.make(c.S, c.N, c.P, 1, 1, 128, max(c.new))

    def __call__(self, stream):
        c = self.c
        logits, tok, par, off, slot, hist, rep, freq, pres, temp, b_off, b_tok, b_val, mask, mrow = c.keep
        G.gdn_logits_probs(self.dm, c.V, c.code, logits, c.stride, tok, par, off, slot, hist, c.stride, rep, freq, pres, temp, b_off, b_tok, b_val,
                           b_tok.numel(), mask, mask.shape[1], mrow, len(mask), self.out, c.ps, c.status, stream=stream)

    def same(self):
        return int(self.c.status) == 0 and torch.equal(self.out, self.want)


class AttnCall:
    def __init__(self, ctx, new, d, tree, seed):
        cache, q, par = case(seed, torch.bfloat16, d, 8, 2, 16, "dense", (1, 1), ctx, new, tree)
        self.a = Attn4(cache, q, ctx, new, par, torch.bfloat16, d ** -0.5)
        self.want = self.a.out()

    def __call__(self, stream):
        self.a(stream=stream)

    def same(self):
        return int(self.a.status) == 0 and torch.equal(self.a.o.cpu(), self.want)


def probs(V, new, seed):
    return ProbsCall(Probs(seed, "bf16", V, new, True).biases([9] * len(new)).masks())


@pytest.mark.parametrize("left,right", [
    (lambda: probs(65536, [16] * 20, 1), lambda: probs(131072, [16] * 6, 2)),                # CTAs that stay, of one and of two a row
    (lambda: probs(131072, [16], 3), lambda: probs(16384, [64] * 5, 4)),
    (lambda: AttnCall([400, 90, 700], [1, 1, 2], 256, False, 5), lambda: AttnCall([300, 20], [16, 40], 128, True, 6)),
    (lambda: AttnCall([500, 3], [30, 7], 256, True, 7), lambda: probs(131072, [16] * 6, 8)),
])
def test_two_streams(left, right):
    calls = [left(), right()]
    streams = [torch.cuda.Stream() for _ in calls]
    torch.cuda.synchronize()
    for _ in range(20):
        for c, s in zip(calls, streams):
            c(s)
    torch.cuda.synchronize()
    assert all(c.same() for c in calls)
