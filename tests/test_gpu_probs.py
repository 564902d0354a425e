"""Logits to probabilities, and the token history's commit, on the GPU against their
64-bit forms.

Tolerance.  x comes out of six fp32 roundings at most, each 2^-24 of an intermediate
value, X at most; then x - max, the quotient by T and the exponent of two are formed in
fp32: an exponent is off by E = (2 * 6 X + 3 (|x - max| + 100 T)) 2^-24 / T, the second
summand also for the terms of the sum that matter (those within 100 T of the largest).
p has one such factor in its numerator and one in its sum, and 2^-20 for the two
exponentials, the product and the sums: |p - ref| <= (2 E + 2^-20) ref, beside 2^-120
where fp32 underflows.  One-hot rows, zeros, counts and marks are exact."""
import numpy as np
import pytest
import torch

import attn_ref as R
import gated_deltanet_speculative_gdn_gb300 as G
import probs_ref as P

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # collected on CPU machines, never run there
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

TYPES = {"bf16": (torch.bfloat16, G.GDN_BF16), "fp16": (torch.float16, G.GDN_FP16), "fp32": (torch.float32, G.GDN_FP32)}


def i32(x):
    return torch.tensor(np.asarray(x, dtype=np.int32), device="cuda")


def f32(x):
    return None if x is None else torch.tensor(np.asarray(x, dtype=np.float32), device="cuda")


def offsets(new):
    return np.concatenate([[0], np.cumsum(new)]).astype(np.int32)


class Probs:
    """One call's inputs on the CPU (changed by a test before the call) and its outcome."""

    def __init__(self, seed, name, V, new, tree=True, slots=None, std=3.0, pad=8):
        rng = self.rng = np.random.default_rng(seed)
        self.dtype, self.code = TYPES[name]
        self.V, self.new, self.N, self.S = V, new, sum(new), len(new)
        self.P = slots or self.S + 2
        self.stride = (V + 7) // 8 * 8 + pad
        self.logits = torch.full((self.N, self.stride), float("nan"), dtype=self.dtype)
        self.logits[:, :V] = torch.tensor(rng.normal(size=(self.N, V)) * std).to(self.dtype)
        self.par = [R.random_tree(rng, k) if tree and k else [i - 1 for i in range(k)] for k in new]
        self.tokens = rng.integers(0, V, self.N).astype(np.int32)
        self.tokens[rng.random(self.N) < 0.5] = rng.integers(0, V)      # one token again and again
        self.slot = rng.permutation(self.P)[:self.S].astype(np.int32)
        self.history = np.zeros((self.P, self.stride), np.uint16)
        some = rng.random((self.P, V)) < 0.05
        self.history[:, :V][some] = rng.integers(1, 6, int(some.sum()))
        self.history[:, :V][rng.random((self.P, V)) < 0.05] |= 0x8000
        self.history[:, V:] = 0xffff
        self.rep, self.freq, self.pres, self.temp = (rng.uniform(lo, hi, self.S).astype(np.float32)
                                                     for lo, hi in ((1.0, 1.5), (-0.3, 0.5), (-0.3, 0.5), (0.5, 1.5)))
        self.bias = self.mask = self.mask_row = None

    def biases(self, counts, std=4.0):
        """Lists of so many distinct tokens for each sequence."""
        self.bias = [[(int(t), np.float32(self.rng.normal() * std)) for t in np.sort(self.rng.permutation(self.V)[:k])] for k in counts]
        return self

    def masks(self, rows=None, share=0.5, pad=1):
        M = self.N if rows is None else max([r for r in rows if r >= 0], default=0) + 1
        words = (self.V + 31) // 32
        bits = self.rng.random((M, words * 32)) < share
        self.mask = np.zeros((M, words + pad), np.uint32)
        self.mask[:, :words] = np.packbits(bits, axis=1, bitorder="little").view(np.uint32)
        self.mask_row = rows
        return self

    def rows(self):
        n = 0
        for s, k in enumerate(self.new):
            for i in range(k):
                yield n, s, i
                n += 1

    def reference(self):
        """[N][V] p, and the tolerance of each."""
        V, off = self.V, offsets(self.new)
        p, tol = np.zeros((self.N, V)), np.zeros((self.N, V))
        has = any(x is not None for x in (self.rep, self.freq, self.pres))
        for n, s, i in self.rows():
            row = self.logits[n, :V].double().numpy()
            hist = self.history[self.slot[s]] if self.history is not None and has else None
            toks = self.tokens[off[s]:off[s + 1]]
            counts, prompt = P.row_counts(hist, toks, self.par[s], i, V) if has else (np.zeros(V, np.int64), np.zeros(V, bool))
            rep, freq, pres, temp = (d if x is None else float(x[s]) for x, d in ((self.rep, 1.0), (self.freq, 0.0), (self.pres, 0.0), (self.temp, 1.0)))
            m = None
            if self.mask is not None:
                r = n if self.mask_row is None else self.mask_row[n]
                m = None if r < 0 else P.allowed_of(self.mask[r], V)
            x = P.adjusted(row, counts, prompt, rep, freq, pres, self.bias[s] if self.bias else [], m)
            p[n] = P.probabilities(x, temp)
            if not temp > 0 or not (x > -np.inf).any() or np.isnan(x).any():
                continue
            fine = np.isfinite(x)
            big = np.abs(row[fine]) * max(rep, 1 / rep) + abs(freq) * counts[fine] + abs(pres)
            if self.bias:
                b = np.zeros(V)
                for t, v in self.bias[s]:
                    b[t] = abs(v)
                big = big + b[fine]
            X = big.max() if len(big) else 0.0
            away = np.where(fine, x.max() - np.where(fine, x, 0), 0.0)
            E = (12 * X + 3 * (away + 100 * temp)) * 2.0 ** -24 / temp
            tol[n] = (2 * E + 2.0 ** -20) * p[n] + 2.0 ** -120
        return p, tol

    def call(self, stream=None, **kw):
        V = self.V
        self.ps = (V + 3) // 4 * 4 + 4
        out = torch.full((self.N, self.ps), 7.0, device="cuda")
        dm = G.GdnDims.make(self.S, self.N, self.P, 1, 1, 128, max([1, *self.new]))
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        b_off = b_tok = b_val = None
        nb = 0
        if self.bias is not None:
            b_off = i32(offsets([len(b) for b in self.bias]))
            flat = [x for b in self.bias for x in b]
            nb = len(flat)
            b_tok, b_val = i32([t for t, _ in flat]), f32([v for _, v in flat])
        mask = None if self.mask is None else torch.from_numpy(self.mask.view(np.int32)).cuda()
        hist = None if self.history is None else torch.from_numpy(self.history.view(np.int16)).cuda()
        self.keep = (self.logits.cuda(), i32(self.tokens), i32([x for p in self.par for x in p]), i32(offsets(self.new)), i32(self.slot), hist,
                     f32(self.rep), f32(self.freq), f32(self.pres), f32(self.temp), b_off, b_tok, b_val, mask,
                     None if self.mask_row is None else i32(self.mask_row))
        a = dict(zip(("logits", "tokens", "parents", "off", "slot", "hist", "rep", "freq", "pres", "temp", "b_off", "b_tok", "b_val", "mask", "mrow"), self.keep))
        a |= dict(nb=nb, nm=0 if self.mask is None else len(self.mask)) | kw
        G.gdn_logits_probs(dm, V, self.code, a["logits"], self.stride, a["tokens"], a["parents"], a["off"], a["slot"], a["hist"], self.stride,
                           a["rep"], a["freq"], a["pres"], a["temp"], a["b_off"], a["b_tok"], a["b_val"], a["nb"], a["mask"],
                           0 if self.mask is None else self.mask.shape[1], a["mrow"], a["nm"], out, self.ps, self.status, stream=stream)
        return out

    def check(self):
        out = self.call().cpu().double().numpy()
        assert int(self.status) == 0
        p, tol = self.reference()
        assert (out[:, self.V:] == 7.0).all()                 # past the vocabulary nothing is written
        got = out[:, :self.V]
        assert np.array_equal(np.isnan(got), np.isnan(p))
        fine = ~np.isnan(p)
        err = np.abs(got - p)[fine]
        assert (err <= tol[fine]).all(), f"largest error / tolerance {float(np.max(err / np.maximum(tol[fine], 1e-300)))}"
        return got


CASES = [
    # dtype, vocab, new, tree, bias counts, mask rows
    ("bf16", 1, [1], True, None, None),
    ("fp16", 7, [3, 0, 2], True, [2, 1, 7], None),
    ("fp32", 33, [5], False, [4], "all"),
    ("bf16", 1000, [16, 1, 0, 40], True, [3, 0, 5, 100], "some"),
    ("fp16", 4099, [9, 64], False, None, "all"),
    ("fp32", 16384, [4], True, [17], None),                       # a slice exactly
    ("bf16", 16392, [4], True, [17], "some"),                     # and one group more
    ("bf16", 50003, [16, 5], True, [40, 300], "some"),
    ("fp32", 131072, [3], True, [5], "all"),
    ("bf16", 262144, [2], False, [9], None),                      # as much as registers hold
    ("fp16", 300007, [2, 1], True, [9, 0], "some"),               # and more: the rest is read again
]


@pytest.mark.parametrize("k", range(len(CASES)))
def test_probabilities(k):
    name, V, new, tree, bias, mask = CASES[k]
    c = Probs(k, name, V, new, tree)
    if bias:
        c.biases(bias)
    if mask == "all":
        c.masks()
    elif mask == "some":
        c.masks([int(c.rng.integers(-1, 3)) for _ in range(c.N)])
    c.check()


def test_many_rows():
    """More rows than the GPU holds at once, odd vocabulary, clusters of several CTAs."""
    c = Probs(50, "bf16", 40001, [16] * 24, True)
    c.temp[5::8] = 0
    c.biases([20] * 24).masks([n if n % 3 else -1 for n in range(c.N)])
    c.check()


ROWS = [
    # dtype, vocab, new: rows that CTAs work through one after the other, one to sixteen CTAs to a row
    ("bf16", 16384, [16] * 21),
    ("fp16", 65536, [16] * 6),
    ("bf16", 65544, [7] * 14),
    ("bf16", 131072, [1] * 90),
    ("fp16", 140001, [16] * 5),
    ("fp32", 32769, [10] * 17),
    ("fp32", 131072, [16] * 4),
    ("bf16", 262144, [16] * 3),
]


@pytest.mark.parametrize("k", range(len(ROWS)))
def test_rows_one_after_the_other(k):
    name, V, new = ROWS[k]
    c = Probs(120 + k, name, V, new, True)
    c.temp[3::7] = 0
    c.biases([(5 * s) % 40 for s in range(c.S)]).masks([n if n % 3 else -1 for n in range(c.N)])
    c.mask[6] = 0                                                 # (row 6 has nothing left)
    c.logits[8, V // 2] = float("nan")
    c.check()


def test_rows_with_errors_between():
    """Rows that are refused, beside others of the same CTAs that are not."""
    V = 131072
    c = Probs(140, "bf16", V, [16] * 10, True)
    c.biases([10] * 10).masks()
    mrow = np.arange(c.N)
    bad = [0, 1, 2, 17, 50, 51, 159]
    mrow[bad] = c.N
    out = c.call(mrow=i32(mrow)).cpu()
    assert int(c.status) == G.GDN_DEV_BAD_MASK
    good = [n for n in range(c.N) if n not in bad]
    ref = c.call().cpu()
    assert int(c.status) == 0
    assert torch.equal(out[good], ref[good]) and bool((out[bad] == 7.0).all())
    one = Probs(140, "bf16", V, [16], True)                       # the same rows by the other kernel
    one.biases([10]).masks()
    for x in ("logits", "tokens"):
        setattr(one, x, getattr(c, x)[:16])
    one.par, one.slot, one.history, one.P, one.mask, one.bias = c.par[:1], c.slot, c.history, c.P, c.mask[:16], c.bias[:1]
    one.rep, one.freq, one.pres, one.temp = c.rep, c.freq, c.pres, c.temp
    again = one.call().cpu()[:, :V].double()
    assert float(((again - ref[:16, :V].double()).abs() / (again + 1e-30)).max()) < 1e-5


@pytest.mark.parametrize("without", ["rep", "freq", "pres", "temp", "history", "penalties", "all"])
def test_parts_left_out(without):
    c = Probs(60, "fp16", 2003, [7, 3], True)
    for x in {"penalties": ("rep", "freq", "pres"), "all": ("rep", "freq", "pres", "temp", "history")}.get(without, (without,)):
        setattr(c, x, None)
    c.check()
    if without == "all":                                          # then none of these is needed
        out = c.call(tokens=None, parents=None, slot=None)
        assert int(c.status) == 0 and torch.equal(out, c.call())


def test_greedy():
    """The largest x, the lowest token among equals, in whatever CTA; the others 0."""
    for V in (9, 5000, 131072):
        c = Probs(70, "fp32", V, [6, 6], False)
        c.history[:] = 0
        c.rep = c.freq = c.pres = None
        c.temp = np.array([0.0, -1.0], np.float32)
        c.logits[:, :V] = torch.randint(-5, 6, (12, V)).float()   # many equal ones
        c.logits[0, V - 1] = 9.0
        c.logits[1, [2, V - 2]] = 9.0
        c.logits[2, :V] = -3.4028234663852886e38                  # all alike, the type's lowest
        c.logits[3, 1] = float("inf")
        c.check()


def test_rows_with_little_left():
    """Masks that leave nothing or one token, infinities and NaN under the mask and beside it, the type's lowest value."""
    for temp in (1.0, 0.0):
        for name, V in (("bf16", 77), ("fp32", 40000)):
            c = Probs(80, name, V, [8], False)
            c.temp = np.array([temp], np.float32)
            c.masks()
            c.mask[0] = 0                                         # nothing
            c.mask[1] = 0
            c.mask[1, 1] = 1 << 5                                 # one token
            low = torch.finfo(c.dtype).min
            c.mask[2:] = 0xffffffff
            c.logits[2, :V] = -float("inf")                       # nothing by the logits themselves
            c.logits[3, :V - 1] = low                             # one token beside the type's lowest (penalised: it stays finite)
            c.logits[4, :V] = low                                 # everything is
            c.mask[5] = 0xfffffffe
            c.logits[5, 0] = float("nan")                         # NaN that the mask forbids
            c.mask[6] = 0xfffffff7
            c.logits[6, 3] = float("inf")                         # and an infinity
            c.logits[7, 2] = float("nan")                         # NaN that it allows
            got = c.check()
            assert (got[0] == 0).all() and got[1, 37] == 1 and (got[2] == 0).all() and np.isnan(got[7]).all()


def test_biases_ban_and_force():
    c = Probs(90, "bf16", 1234, [4], True)
    c.bias = [[(0, np.float32(-np.inf)), (7, np.float32(50.0)), (8, np.float32(-np.inf)), (1233, np.float32(0.5))]]
    got = c.check()
    assert (got[:, [0, 8]] == 0).all() and (got[:, 7] > 0.5).all()


def test_extreme_temperatures():
    for t in (1e-38, 1e-45, 1e30, float("inf")):
        c = Probs(95, "fp32", 300, [3], True)
        c.rep = c.freq = c.pres = None
        c.logits[:, :300] = torch.randint(-3, 4, (3, 300)).float()
        c.logits[:, 5] = 4.0
        c.masks()
        c.mask[:, 0] |= 1 << 5
        c.temp = np.array([t], np.float32)
        got = c.call().cpu().double().numpy()[:, :300]
        for n in range(3):
            ok = P.allowed_of(c.mask[n], 300)
            if t < 1:
                want = (np.arange(300) == 5).astype(float)
            else:
                want = ok / ok.sum()
            assert np.allclose(got[n], want, rtol=1e-6, atol=0)


def test_counts_stop():
    """A count at its end stays there, with the prompt's mark; the path's tokens add to it."""
    c = Probs(97, "fp32", 64, [40], False)
    c.rep = c.pres = None
    c.freq = np.array([2.0 ** -12], np.float32)
    c.tokens[:] = 3
    c.history[:, :64] = 0
    c.history[c.slot[0], 3] = 0x8000 | (0x7fff - 10)
    c.check()


def test_device_errors():
    c = Probs(98, "bf16", 500, [4, 4], True)
    c.biases([3, 3]).masks([0, 1, 2, 3, 0, 1, 2, 3])
    flat = [x for p in c.par for x in p]
    bad_slot = c.slot.copy()
    bad_slot[1] = c.P
    tok = c.tokens.copy()
    tok[4] = 500                                                  # sequence 1's root
    b = [t for x in c.bias for t, _ in x]
    for code, kw in ((G.GDN_DEV_BAD_NODE_OFF, dict(off=i32([0, 4, 7]))), (G.GDN_DEV_BAD_NODE_OFF, dict(off=i32([1, 4, 8]))),
                     (G.GDN_DEV_BAD_PARENT, dict(parents=i32(flat[:5] + [1] + flat[6:]))), (G.GDN_DEV_BAD_PARENT, dict(parents=i32([-2] + flat[1:]))),
                     (G.GDN_DEV_BAD_SLOT, dict(slot=i32(bad_slot))), (G.GDN_DEV_BAD_SLOT, dict(slot=i32([-1, 0]))),
                     (G.GDN_DEV_BAD_TOKEN, dict(tokens=i32(tok))), (G.GDN_DEV_BAD_TOKEN, dict(b_tok=i32(b[:5] + [500]))),
                     (G.GDN_DEV_BAD_TOKEN, dict(b_tok=i32([b[0], b[0], b[2]] + b[3:]))), (G.GDN_DEV_BAD_BIAS, dict(b_off=i32([0, 3, 7]))),
                     (G.GDN_DEV_BAD_BIAS, dict(b_off=i32([0, 3, 2]))), (G.GDN_DEV_BAD_BIAS, dict(b_off=i32([-1, 3, 6]))),
                     (G.GDN_DEV_BAD_MASK, dict(mrow=i32([0, 1, 2, 4, 0, 1, 2, 3]))), (G.GDN_DEV_BAD_MASK, dict(mrow=i32([0, 1, 2, 3, -2, 1, 2, 3])))):
        out = c.call(**kw)
        assert int(c.status) == code, (kw, int(c.status), code)
        rows = (out != 7.0).any(1)
        assert not rows.all()                                     # the rows that the error reaches are not written
    c.check()


def test_equal_calls_and_streams():
    """Twice the same bits, on another stream, and in a graph."""
    c = Probs(99, "bf16", 131072, [16] * 3, True)
    c.biases([10] * 3).masks()
    a = c.call()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        b = c.call()
    torch.cuda.synchronize()
    assert torch.equal(a, b) and int(c.status) == 0


@pytest.mark.parametrize("V,new", [(131072, [16] * 32), (131072, [16] * 3), (1000, [5, 0, 64, 1])])
def test_in_a_graph(V, new):
    """A captured call sees the inputs of each replay, and gives the bits of a plain call."""
    c = Probs(7, "bf16", V, new, True)
    a = Probs(8, "bf16", V, new, True)
    want = [x.call() for x in (c, a)]
    dims = G.GdnDims.make(c.S, c.N, c.P, 1, 1, 128, max(new))
    x = [t.clone() for t in c.keep[:10]]
    out = torch.zeros(c.N, c.stride, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        G.gdn_logits_probs(dims, V, c.code, x[0], c.stride, *x[1:6], c.stride, *x[6:], None, None, None, 0, None, 0, None, 0, out, c.stride, st)
    for k in (0, 1, 0):
        for t, y in zip(x, (c, a)[k].keep):
            t.copy_(y)
        g.replay()
        torch.cuda.synchronize()
        assert int(st) == 0 and torch.equal(out[:, :V].cpu(), want[k][:, :V].cpu())


# ---- the history's commit ---------------------------------------------------------------


def commit(c_dims, V, tokens, acc, par, off, slot, prompt, hist, st):
    G.gdn_token_commit(c_dims, V, tokens, acc, par, off, slot, prompt, hist, hist.stride(0), st)
    torch.cuda.synchronize()


@pytest.mark.parametrize("V", [5, 1000, 131072])
def test_token_commit(V):
    rng = np.random.default_rng(V)
    new = [16, 0, 64, 1, 33]
    S, N, slots, stride = len(new), sum(new), 8, (V + 7) // 8 * 8 + 8
    par = [R.random_tree(rng, k) if k else [] for k in new]
    par[2] = [i - 1 for i in range(64)]
    acc = [int(rng.integers(0, k)) if k else -1 for k in new]
    acc[2], acc[3] = 63, -1
    tokens = rng.integers(0, V, N).astype(np.int32)
    tokens[16:50] = V - 1                                         # one token 34 times in a path
    slot = rng.permutation(slots)[:S].astype(np.int32)
    h = rng.integers(0, 1 << 16, (slots, stride)).astype(np.uint16)
    h[slot[2], V - 1] = 0x7fff - 3
    dm = G.GdnDims.make(S, N, slots, 1, 1, 128, 64)
    hist, st = torch.from_numpy(h.view(np.int16)).cuda(), torch.zeros(1, dtype=torch.int32, device="cuda")
    commit(dm, V, i32(tokens), i32(acc), i32([x for p in par for x in p]), i32(offsets(new)), i32(slot), 0, hist, st)
    assert int(st) == 0
    want, n0 = h.copy(), 0
    for s, k in enumerate(new):
        for x in R.path_of(par[s], acc[s]):
            e = want[slot[s], tokens[n0 + x]]
            want[slot[s], tokens[n0 + x]] = (e & 0x8000) | min((e & 0x7fff) + 1, 0x7fff)
        n0 += k
    assert np.array_equal(hist.cpu().numpy().view(np.uint16), want)


@pytest.mark.parametrize("prompt", [0, 1])
def test_token_commit_of_prompts(prompt):
    """All tokens of sequences of any length, marked or counted."""
    rng = np.random.default_rng(prompt)
    V, new, slots = 777, [3000, 1, 0, 258], 5
    S, N, stride = len(new), sum(new), 784
    tokens = rng.integers(0, V, N).astype(np.int32)
    tokens[::2] = tokens[0]
    slot = np.array([4, 0, 4, 2], np.int32)                       # the empty sequence may share a slot
    h = np.zeros((slots, stride), np.uint16)
    h[:, :V] = rng.integers(0, 3, (slots, V))
    dm = G.GdnDims.make(S, N, slots, 1, 1, 128, 1)
    hist, st = torch.from_numpy(h.view(np.int16)).cuda(), torch.zeros(1, dtype=torch.int32, device="cuda")
    commit(dm, V, i32(tokens), None, None, i32(offsets(new)), i32(slot), prompt, hist, st)
    assert int(st) == 0
    want, n = h.copy(), 0
    for s, k in enumerate(new):
        for t in tokens[n:n + k]:
            if prompt:
                want[slot[s], t] |= 0x8000
            else:
                want[slot[s], t] += 1
        n += k
    assert np.array_equal(hist.cpu().numpy().view(np.uint16), want)


def test_token_commit_errors_write_nothing():
    V, slots = 100, 4
    dm = G.GdnDims.make(2, 8, slots, 1, 1, 128, 4)
    h = torch.zeros(slots, 104, dtype=torch.int16, device="cuda")
    good = dict(tok=[1, 2, 3, 4, 5, 6, 7, 8], acc=[3, 3], par=[-1, 0, 1, 2] * 2, off=[0, 4, 8], slot=[1, 2])
    for code, kw in ((G.GDN_DEV_BAD_NODE_OFF, dict(off=[0, 4, 9])), (G.GDN_DEV_BAD_NODE_OFF, dict(off=[0, 3, 8])), (G.GDN_DEV_BAD_ACCEPTED, dict(acc=[4, 0])),
                     (G.GDN_DEV_BAD_ACCEPTED, dict(acc=[-2, 0])), (G.GDN_DEV_BAD_PARENT, dict(par=[-1, 0, 1, 3] + [-1, 0, 1, 2])),
                     (G.GDN_DEV_BAD_SLOT, dict(slot=[1, 4])), (G.GDN_DEV_BAD_SLOT, dict(slot=[-1, 2])), (G.GDN_DEV_DUP_SLOT, dict(slot=[2, 2])),
                     (G.GDN_DEV_BAD_TOKEN, dict(tok=[1, 2, 3, 100, 5, 6, 7, 8])), (G.GDN_DEV_BAD_TOKEN, dict(tok=[1, 2, 3, 4, -1, 6, 7, 8]))):
        a = good | kw
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        commit(dm, V, i32(a["tok"]), i32(a["acc"]), i32(a["par"]), i32(a["off"]), i32(a["slot"]), 0, h, st)
        assert int(st) == code, (kw, int(st))
        assert not h.any()
    st.fill_(G.GDN_DEV_TIMEOUT)
    commit(dm, V, i32(good["tok"]), i32(good["acc"]), i32(good["par"]), i32(good["off"]), i32(good["slot"]), 0, h, st)
    assert not h.any()
    # a token off the accepted path is not looked at
    st.zero_()
    commit(dm, V, i32([1, 2, 3, 1 << 30, 5, 6, 7, 8]), i32([2, -1]), i32(good["par"]), i32(good["off"]), i32([1, 99]), 0, h, st)
    assert int(st) == 0 and h.sum() == 3


@pytest.mark.parametrize("at", [0, 300, 4000])
def test_token_commit_errors_anywhere_in_a_prompt(at):
    """One bad token among several CTAs' shares of a long prompt: nothing of any sequence is written."""
    V, new = 100, [5, 4001]
    tokens = np.arange(sum(new)) % V
    tokens[5 + at] = V
    dm = G.GdnDims.make(2, sum(new), 2, 1, 1, 128, 1)
    hist, st = torch.zeros(2, 104, dtype=torch.int16, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    commit(dm, V, i32(tokens), None, None, i32(offsets(new)), i32([1, 0]), 1, hist, st)
    assert int(st) == G.GDN_DEV_BAD_TOKEN and not hist.any()
