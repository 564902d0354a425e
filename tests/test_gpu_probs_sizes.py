"""gdn_logits_probs at the sizes where its kernels take another form: rows of 8 and 16 CTAs one after the other, and
vocabularies of which registers hold the first 262,144 tokens and the rest is read again for every pass.

Tolerances: those of test_gpu_probs.py."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # collected on CPU machines, never run there
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import gated_deltanet_speculative_gdn_gb300 as G  # noqa: E402
import probs_ref as P  # noqa: E402
from test_gpu_probs import Probs  # noqa: E402

ROWS = [
    # dtype, vocab, new; CTAs to a row
    ("fp32", 151936, [16] * 4),      # 8
    ("bf16", 270001, [11] * 3),      # 8
    ("bf16", 151936, [16] * 2),      # 4
    ("fp32", 300007, [12] * 2),      # 16
    ("fp16", 600001, [10, 0, 12]),   # 16
    ("bf16", 40001, [16] * 24),      # 1
]


@pytest.mark.parametrize("k", range(len(ROWS)))
def test_rows_of_many_ctas(k):
    name, V, new = ROWS[k]
    c = Probs(160 + k, name, V, new, True)
    c.temp[::2] = 0
    c.biases([(7 * s + 3) % 40 for s in range(c.S)]).masks([n if n % 3 else -1 for n in range(c.N)])
    c.mask[4] = 0                                                 # (nothing is left of row 4, nor of the last)
    c.logits[c.N - 1, :V] = -float("inf")
    c.logits[8, V - 1], c.logits[c.N - 2, 5] = float("nan"), float("nan")
    c.mask[8] = 0xffffffff
    got = c.check()
    assert (got[[4, c.N - 1]] == 0).all()
    assert np.isnan(got[8]).all()


REST = 262144
V = 300007


def test_greedy_among_tokens_that_are_read_again():
    c = Probs(170, "fp32", V, [6, 6], False)
    c.history[:] = 0
    c.rep = c.freq = c.pres = None
    c.temp = np.array([0.0, -1.0], np.float32)
    c.logits[:, :V] = torch.randint(-5, 6, (12, V)).float()
    c.logits[0, V - 1] = 9.0
    c.logits[1, [REST + 4, V - 2]] = 9.0
    c.logits[2, [REST - 1, REST]] = 9.0
    c.logits[3, [17, V - 9]] = 9.0
    c.logits[4, :V] = -3.4028234663852886e38                      # all alike, the type's lowest
    c.logits[5, REST + 1000] = float("inf")
    c.logits[6, :V] = -float("inf")
    c.logits[6, REST + 77] = -1e38
    c.logits[7, :V] = -float("inf")
    c.logits[8, V - 3] = float("nan")
    c.check()


@pytest.mark.parametrize("temp", [1.0, 0.0])
@pytest.mark.parametrize("name", ["bf16", "fp32"])
def test_rows_with_little_left_in_what_is_read_again(name, temp):
    c = Probs(171, name, V, [8], False)
    c.temp = np.array([temp], np.float32)
    c.masks()
    c.mask[:2] = 0                                                # nothing; one token
    c.mask[1, (V - 1) // 32] = 1 << ((V - 1) % 32)
    low = torch.finfo(c.dtype).min
    c.mask[2:] = 0xffffffff
    c.logits[2, :V] = -float("inf")
    c.logits[3, :V] = low
    c.logits[3, REST + 3] = 1.0
    c.logits[4, :V] = low
    c.mask[5, (REST + 64) // 32] = 0xfffffffe
    c.logits[5, REST + 64] = float("nan")                         # NaN that the mask forbids
    c.mask[6, (V - 2) // 32] = 0xffffffff ^ (1 << ((V - 2) % 32))
    c.logits[6, V - 2] = float("inf")                             # and an infinity
    c.logits[7, REST + 9] = float("nan")                          # NaN that it allows
    got = c.check()
    assert (got[0] == 0).all() and got[1, V - 1] == 1 and (got[2] == 0).all() and np.isnan(got[7]).all()


@pytest.mark.parametrize("V,new", [(16384, [64] * 5), (V, [3])])
@pytest.mark.parametrize("t", [1e-38, 1e-45, 1e30, float("inf")])
def test_extreme_temperatures(t, V, new):
    """As in test_gpu_probs.py, for many rows and for what is read again."""
    c = Probs(172, "fp32", V, new, False)
    c.rep = c.freq = c.pres = None
    c.logits[:, :V] = torch.randint(-3, 4, (c.N, V)).float()
    top = V - 7
    c.logits[:, top] = 4.0
    c.masks([0] * c.N)
    c.mask[:, top // 32] |= np.uint32(1 << (top % 32))
    c.temp = np.full(c.S, t, np.float32)
    got = c.call().cpu().double().numpy()[:, :V]
    ok = P.allowed_of(c.mask[0], V)
    want = (np.arange(V) == top).astype(float) if t < 1 else ok / ok.sum()
    assert int(c.status) == 0 and np.allclose(got, want, rtol=1e-6, atol=0)


@pytest.mark.parametrize("V,new,far", [(5000, [3, 1], 1 << 30), (16384, [64] * 5, 1 << 24)])
def test_far_rows(V, new, far):
    """Rows of logits, probabilities, history and masks whose places pass 2^32 elements: the bits of dense ones."""
    c = Probs(173, "bf16", V, new, True, slots=len(new))
    c.biases([9] * c.S).masks()
    dense = c.call()
    logits, _, _, _, _, hist, _, _, _, _, _, _, _, mask, _ = c.keep
    assert int(c.status) == 0

    def spread(x, stride):
        y = torch.empty((len(x) - 1) * stride + x.shape[1], dtype=x.dtype, device="cuda")
        y.as_strided(x.shape, (stride, 1)).copy_(x)
        return y

    masks = far // 8                                              # (words of 32 tokens)
    p = torch.full(((c.N - 1) * far + c.ps,), 7.0, device="cuda")
    dm = G.GdnDims.make(c.S, c.N, c.P, 1, 1, 128, max(new))
    _, tok, par, off, slot, _, rep, freq, pres, temp, b_off, b_tok, b_val, _, _ = c.keep
    G.gdn_logits_probs(dm, V, c.code, spread(logits, far), far, tok, par, off, slot, spread(hist, far), far, rep, freq, pres, temp, b_off, b_tok, b_val,
                       b_tok.numel(), spread(mask, masks), masks, None, c.N, p, far, c.status)
    assert int(c.status) == 0 and torch.equal(p.as_strided(dense.shape, (far, 1)), dense)
    h = torch.zeros((c.P - 1) * far + c.stride, dtype=torch.int16, device="cuda")
    G.gdn_token_commit(dm, V, tok, None, None, off, slot, 0, h, far, c.status)
    assert int(c.status) == 0
    want = np.zeros((c.P, c.stride), np.int16)
    np.add.at(want, (c.slot.repeat(new), c.tokens), 1)
    assert np.array_equal(h.as_strided((c.P, c.stride), (far, 1)).cpu().numpy(), want)
