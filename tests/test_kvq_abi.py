"""Host-side refusals of the 4-bit cache's and of the sampling's entry points (CPU: no kernel is
launched), and checks of the 64-bit forms that the GPU tests use."""
import numpy as np
import pytest
import torch

import gated_deltanet_speculative_gdn_gb300 as G
import kv4_ref as Q
import probs_ref as P

FAKE = 1 << 24          # 16-byte aligned, never dereferenced


def dims(**kw):
    base = dict(n_seqs=2, n_tokens=8, max_seq_tokens=8, h_q=4, h_kv=2, d_head=64, dtype=G.GDN_BF16, n_pages=8,
                page_size=16, table_width=4)
    base.update(kw)
    return G.AttnDims.make_kvq(**base)


def append(d, **kw):
    w = d.h_kv * d.d_head
    a = dict(k=FAKE, ks=w, v=2 * FAKE, vs=w, ku=1.0, vu=1.0, off=3 * FAKE, ctx=4 * FAKE, table=5 * FAKE, kp=6 * FAKE, vp=7 * FAKE, status=8 * FAKE)
    a.update(kw)
    return G.gdn_kvq_append(d, a["k"], a["ks"], a["v"], a["vs"], a["ku"], a["vu"], a["off"], a["ctx"], a["table"], a["kp"], a["vp"],
                            a["status"], stream=0, raise_on_error=False)


def read(d, **kw):
    a = dict(layers=1, ls=0, kp=FAKE, vp=2 * FAKE, ku=1.0, vu=1.0, off=3 * FAKE, ctx=4 * FAKE, table=5 * FAKE, k=6 * FAKE, v=7 * FAKE,
             rs=d.h_kv * d.d_head, status=8 * FAKE)
    a.update(kw)
    return G.gdn_kvq_read(d, a["layers"], a["ls"], a["kp"], a["vp"], a["ku"], a["vu"], a["off"], a["ctx"], a["table"], a["k"], a["v"], a["rs"],
                          a["status"], stream=0, raise_on_error=False)


def attend(d, **kw):
    a = dict(q=FAKE, qs=d.h_q * d.d_head, kp=2 * FAKE, vp=3 * FAKE, ku=1.0, vu=1.0, table=4 * FAKE, ctx=5 * FAKE, off=6 * FAKE, par=None,
             scale=0.125, o=8 * FAKE, ws=64 * FAKE, wb=1 << 40, status=10 * FAKE)
    a.update(kw)
    return G.gdn_paged_attention_kvq(d, a["q"], a["qs"], a["kp"], a["vp"], a["ku"], a["vu"], a["table"], a["ctx"], a["off"], a["par"], a["scale"],
                                     a["o"], a["ws"], a["wb"], a["status"], stream=0, raise_on_error=False)


def move(d, **kw):
    a = dict(layers=2, ls=1 << 16, acc=FAKE, par=2 * FAKE, off=3 * FAKE, ctx=4 * FAKE, table=5 * FAKE, kp=6 * FAKE,
             vp=7 * FAKE, nl=8 * FAKE, status=9 * FAKE)
    a.update(kw)
    return G.gdn_kvq_commit(d, a["layers"], a["ls"], a["acc"], a["par"], a["off"], a["ctx"], a["table"], a["kp"], a["vp"],
                            a["nl"], a["status"], stream=0, raise_on_error=False)


def probs(d=None, **kw):
    d = d or G.GdnDims.make(2, 8, 4, 1, 1, 16, 16)
    a = dict(vocab=100, dtype=G.GDN_BF16, logits=FAKE, ls=104, tok=2 * FAKE, par=3 * FAKE, off=4 * FAKE, slot=5 * FAKE, hist=6 * FAKE, hs=104,
             rep=7 * FAKE, freq=8 * FAKE, pres=9 * FAKE, temp=10 * FAKE, boff=11 * FAKE, btok=12 * FAKE, bval=13 * FAKE, nb=6, mask=14 * FAKE, ms=4,
             mrow=15 * FAKE, nm=3, p=16 * FAKE, ps=100, status=17 * FAKE)
    a.update(kw)
    return G.gdn_logits_probs(d, a["vocab"], a["dtype"], a["logits"], a["ls"], a["tok"], a["par"], a["off"], a["slot"], a["hist"], a["hs"], a["rep"],
                              a["freq"], a["pres"], a["temp"], a["boff"], a["btok"], a["bval"], a["nb"], a["mask"], a["ms"], a["mrow"], a["nm"],
                              a["p"], a["ps"], a["status"], stream=0, raise_on_error=False)


def tokens(d=None, **kw):
    d = d or G.GdnDims.make(2, 8, 4, 1, 1, 16, 16)
    a = dict(vocab=100, tok=FAKE, acc=2 * FAKE, par=3 * FAKE, off=4 * FAKE, slot=5 * FAKE, prompt=0, hist=6 * FAKE, hs=104, status=7 * FAKE)
    a.update(kw)
    return G.gdn_token_commit(d, a["vocab"], a["tok"], a["acc"], a["par"], a["off"], a["slot"], a["prompt"], a["hist"], a["hs"], a["status"],
                              stream=0, raise_on_error=False)


@pytest.mark.parametrize("bad", [
    dict(d_head=96), dict(h_q=3), dict(h_kv=0), dict(h_q=258, h_kv=2), dict(dtype=G.GDN_FP32), dict(n_pages=0), dict(page_size=24),
    dict(page_size=4), dict(page_size=2048), dict(table_width=0), dict(n_seqs=-1), dict(n_tokens=-1), dict(max_seq_tokens=0),
    dict(table_width=1 << 28)])
def test_bad_dims(bad):
    d = dims(page_stride=1 << 20, head_stride=1 << 18, **bad)
    assert append(d) == read(d) == attend(d) == move(d) == G.GDN_ERR_DIMS
    assert G.gdn_attention_kvq_workspace_bytes(d) == G.gdn_kvq_block_bytes(d) == 0


def test_strides():
    block = G.gdn_kvq_block_bytes(dims())
    assert block == 16 * 64 * 9 // 16
    for bad in (dict(page_stride=block - 16), dict(head_stride=block - 16), dict(head_stride=block + 8), dict(page_stride=-block), dict(page_stride=0)):
        d = dims(**bad)
        assert append(d) == read(d) == attend(d) == move(d) == G.GDN_ERR_STRIDE
    d = dims()
    assert append(d, ks=120) == append(d, vs=132) == read(d, rs=120) == attend(d, qs=252) == G.GDN_ERR_STRIDE
    assert read(d, layers=2, ls=-16) == read(d, layers=2, ls=8) == move(d, ls=24) == G.GDN_ERR_STRIDE
    # layers that share blocks
    assert move(d, layers=2, ls=2 * block) == move(d, layers=3, ls=16 * block - 16) == G.GDN_ERR_STRIDE
    assert move(dims(page_stride=3 * block, head_stride=24 * block), layers=4, ls=block) == G.GDN_ERR_STRIDE


def test_units():
    d = dims()
    for u in (0.0, -1.0, 3.0, 2.0 ** 25, 2.0 ** -25, float("inf"), float("nan")):
        for name in ("ku", "vu"):
            assert append(d, **{name: u}) == read(d, **{name: u}) == attend(d, **{name: u}) == G.GDN_ERR_ARG


def test_nulls_and_empty_batches():
    d = dims()
    for call, names in ((append, ("k", "v", "off", "ctx", "table", "kp", "vp", "status")), (read, ("k", "v", "off", "ctx", "table", "kp", "vp", "status")),
                        (attend, ("q", "kp", "vp", "table", "ctx", "off", "o", "ws", "status")),
                        (move, ("acc", "par", "off", "ctx", "table", "kp", "vp", "nl", "status"))):
        for name in names:
            assert call(d, **{name: None}) == G.GDN_ERR_NULL, (call, name)
    for name in ("logits", "off", "p", "status", "tok", "par", "slot", "boff", "btok", "bval"):
        assert probs(**{name: None}) == G.GDN_ERR_NULL, name
    for name in ("tok", "par", "off", "slot", "hist", "status"):
        assert tokens(**{name: None}) == G.GDN_ERR_NULL, name
    for e in (dims(n_seqs=0, n_tokens=0), dims(n_tokens=0)):
        assert append(e, k=None) == read(e, k=None) == attend(e, q=None) == G.GDN_OK
    assert read(d, layers=0) == move(d, layers=0) == move(dims(n_seqs=0, n_tokens=0), acc=None) == G.GDN_OK
    for e in (G.GdnDims.make(0, 0, 1, 1, 1, 16, 16), G.GdnDims.make(2, 0, 1, 1, 1, 16, 16)):
        assert probs(e, logits=None) == tokens(e, tok=None) == G.GDN_OK


def test_alignment_and_overlaps():
    d = dims()
    assert append(d, k=FAKE + 8) == append(d, vp=7 * FAKE + 4) == read(d, v=7 * FAKE + 2) == attend(d, o=8 * FAKE + 8) == G.GDN_ERR_ALIGN
    assert append(d, kp=FAKE) == append(d, vp=2 * FAKE + 64) == append(d, kp=5 * FAKE) == read(d, k=FAKE) == read(d, v=6 * FAKE) == G.GDN_ERR_ALIAS
    assert read(d, v=6 * FAKE + 64) == attend(d, o=FAKE) == attend(d, ws=3 * FAKE) == move(d, nl=6 * FAKE) == move(d, nl=4 * FAKE) == G.GDN_ERR_ALIAS
    assert move(d, vp=FAKE) == probs(p=FAKE) == probs(p=6 * FAKE) == probs(p=14 * FAKE) == tokens(hist=FAKE) == G.GDN_ERR_ALIAS
    assert probs(logits=FAKE + 8) == probs(p=16 * FAKE + 4) == probs(hist=6 * FAKE + 2) == tokens(hist=6 * FAKE + 2) == G.GDN_ERR_ALIGN


def test_arguments():
    d = dims()
    assert attend(d, wb=G.gdn_attention_kvq_workspace_bytes(d) - 1) == attend(d, wb=-1) == G.GDN_ERR_ARG
    for s in (0.0, -1.0, float("nan"), float("inf")):
        assert attend(d, scale=s) == G.GDN_ERR_ARG
    assert attend(dims(max_seq_tokens=65), par=FAKE * 7) == move(dims(max_seq_tokens=65)) == G.GDN_ERR_DIMS
    assert read(d, layers=-1) == move(d, layers=-1) == read(d, layers=65536) == move(d, layers=65536) == G.GDN_ERR_ARG
    for v in (0, -1, (1 << 28) + 1):
        assert probs(vocab=v) == tokens(vocab=v) == G.GDN_ERR_ARG
    assert probs(dtype=3) == probs(dtype=-1) == probs(nb=-1) == probs(nm=-1) == tokens(prompt=2) == G.GDN_ERR_ARG
    assert probs(ls=96) == probs(ls=108) == probs(hs=96) == probs(ps=96) == probs(ps=102) == probs(ms=3) == G.GDN_ERR_STRIDE
    assert tokens(hs=100) == tokens(hs=96) == G.GDN_ERR_STRIDE
    assert probs(G.GdnDims.make(2, 8, 4, 1, 1, 16, 65)) == tokens(G.GdnDims.make(2, 8, 4, 1, 1, 16, 0)) == G.GDN_ERR_DIMS


def test_scale_times_unit():
    """The keys' unit multiplies the scale: both in range, their product not."""
    assert attend(dims(), scale=1e32, ku=2.0 ** 24) == attend(dims(), scale=2e38, ku=1.0) == G.GDN_ERR_ARG
    assert attend(dims(n_tokens=0), scale=1e32, ku=2.0 ** -24) == attend(dims(n_tokens=0), scale=1e30, ku=2.0 ** 24) == G.GDN_OK


def test_nearest_codes_are_nearest():
    """The reference's codes against a plain search over all values, ties to the even code by hand."""
    for grid in (Q.E2M1, Q.E4M3):
        x = torch.cat([torch.rand(2000, dtype=torch.float64) * float(grid[-1]) * 1.2, grid, torch.tensor([1e9, float("inf")])])
        i = Q.nearest_code(grid, x)
        d = (x[:, None] - grid[None]).abs()
        ok = torch.isinf(x) | (d.gather(1, i[:, None])[:, 0] == d.min(1).values)
        assert bool(ok.all())
    ties = {0.25: 0, 0.75: 2, 1.25: 2, 1.75: 4, 2.5: 4, 3.5: 6, 5.0: 6}
    assert Q.nearest_code(Q.E2M1, torch.tensor(list(ties), dtype=torch.float64)).tolist() == list(ties.values())
    assert torch.equal(Q.E4M3, torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double())


def test_quantise_by_hand():
    """One block: the largest of 12 gives the scale 2; the others in steps of that."""
    x = torch.zeros(1, 16, dtype=torch.float64)
    x[0, :6] = torch.tensor([12.0, -1.0, 0.4, 5.0, -7.0, 9.9])       # / 2: 6, -.5, .2, 2.5, -3.5, 4.95
    c, s = Q.quantise(x, 1.0)
    assert s.tolist() == [[0x40]]                                    # 2.0 in e4m3
    assert Q.values(c, s, 1.0)[0, :6].tolist() == [12.0, -1.0, 0.0, 4.0, -8.0, 8.0]
    assert c[0, 0].item() == 7 | (9 << 4)


def test_probabilities_by_hand():
    x = P.adjusted(np.array([2.0, -2.0, 1.0, 4.0]), np.array([1, 2, 0, 0]), np.array([False, False, True, False]), 2.0, 0.5, 0.25, [(3, -1.0)],
                   np.array([True, True, True, True]))
    assert x.tolist() == [2 / 2 - 0.5 - 0.25, -4 - 1.0 - 0.25, 0.5, 3.0]
    assert P.probabilities(np.array([0.0, np.log(3.0)]), 1.0) == pytest.approx([0.25, 0.75])
    assert P.probabilities(np.array([1.0, 5.0, 5.0]), 0.0).tolist() == [0, 1, 0]
    assert P.probabilities(np.array([-np.inf, -np.inf]), 1.0).tolist() == [0, 0]
