"""Host-side refusals of the attention-layer and acceptance entry points (CPU: no
kernel is launched), and checks of their 64-bit forms against closed forms."""
import math

import numpy as np
import pytest
import torch

import attn_ref as R
import gated_deltanet_speculative_gdn_gb300 as G

FAKE = 1 << 24          # 16-byte aligned, never dereferenced


def dims(**kw):
    base = dict(n_seqs=2, n_tokens=8, max_seq_tokens=8, h_q=4, h_kv=2, d_head=64, dtype=G.GDN_BF16, n_pages=8,
                page_size=16, table_width=4)
    base.update(kw)
    return G.AttnDims.make(**base)


def rope(d, **kw):
    a = dict(q=FAKE, qs=d.h_q * d.d_head, k=2 * FAKE, ks=d.h_kv * d.d_head, v=3 * FAKE, vs=d.h_kv * d.d_head, qw=4 * FAKE,
             kw=5 * FAKE, eps=1e-6, pos=6 * FAKE, n_axes=1, inv_freq=7 * FAKE, axis=8 * FAKE, rot=32, inter=0, off=9 * FAKE,
             ctx=10 * FAKE, table=11 * FAKE, qo=12 * FAKE, qos=d.h_q * d.d_head, kp=13 * FAKE, vp=14 * FAKE,
             status=15 * FAKE)
    a.update(kw)
    return G.gdn_rope_append(d, a["q"], a["qs"], a["k"], a["ks"], a["v"], a["vs"], a["qw"], a["kw"], a["eps"], a["pos"],
                             a["n_axes"], a["inv_freq"], a["axis"], a["rot"], a["inter"], a["off"], a["ctx"], a["table"],
                             a["qo"], a["qos"], a["kp"], a["vp"], a["status"], stream=0, raise_on_error=False)


def attend(d, **kw):
    a = dict(q=FAKE, qs=d.h_q * d.d_head, kp=2 * FAKE, vp=3 * FAKE, table=4 * FAKE, ctx=5 * FAKE, off=6 * FAKE, par=None,
             scale=0.125, o=8 * FAKE, ws=64 * FAKE, wb=1 << 40, status=10 * FAKE)
    a.update(kw)
    return G.gdn_paged_attention(d, a["q"], a["qs"], a["kp"], a["vp"], a["table"], a["ctx"], a["off"], a["par"], a["scale"],
                                 a["o"], a["ws"], a["wb"], a["status"], stream=0, raise_on_error=False)


def move(d, **kw):
    a = dict(layers=2, ls=1 << 16, acc=FAKE, par=2 * FAKE, off=3 * FAKE, ctx=4 * FAKE, table=5 * FAKE, kp=6 * FAKE,
             vp=7 * FAKE, nl=8 * FAKE, status=9 * FAKE)
    a.update(kw)
    return G.gdn_kv_commit(d, a["layers"], a["ls"], a["acc"], a["par"], a["off"], a["ctx"], a["table"], a["kp"], a["vp"],
                           a["nl"], a["status"], stream=0, raise_on_error=False)


def accept(d=None, **kw):
    d = d or G.GdnDims.make(2, 8, 1, 1, 1, 16, 16)
    a = dict(vocab=100, p=FAKE, ps=100, q=2 * FAKE, qs=100, rep=0, tok=3 * FAKE, par=4 * FAKE, off=5 * FAKE, u=6 * FAKE,
             un=7 * FAKE, acc=8 * FAKE, nt=9 * FAKE, na=10 * FAKE, status=11 * FAKE)
    a.update(kw)
    return G.gdn_tree_accept(d, a["vocab"], a["p"], a["ps"], a["q"], a["qs"], a["rep"], a["tok"], a["par"], a["off"], a["u"],
                             a["un"], a["acc"], a["nt"], a["na"], a["status"], stream=0, raise_on_error=False)


@pytest.mark.parametrize("bad", [
    dict(d_head=96), dict(h_q=3), dict(h_kv=0), dict(h_q=1), dict(h_q=258, h_kv=2), dict(dtype=2), dict(n_pages=0),
    dict(page_size=24), dict(page_size=4), dict(page_size=2048), dict(table_width=0), dict(n_seqs=-1), dict(n_tokens=-1),
    dict(max_seq_tokens=0), dict(table_width=1 << 28)])
def test_bad_dims(bad):
    base = dict(n_seqs=2, n_tokens=8, max_seq_tokens=8, h_q=4, h_kv=2, d_head=64, dtype=0, n_pages=8, page_size=16,
                table_width=4)
    base.update(bad)
    d = G.AttnDims.make(page_stride=1 << 14, token_stride=1 << 9, head_stride=256, **base)
    assert rope(d, rot=0) == attend(d) == move(d) == G.GDN_ERR_DIMS
    assert G.gdn_attention_workspace_bytes(d) == 0


@pytest.mark.parametrize("bad", [dict(page_stride=1020), dict(token_stride=60), dict(head_stride=68), dict(head_stride=-64)])
def test_bad_cache_strides(bad):
    d = dims(**bad)
    assert rope(d) == attend(d) == move(d) == G.GDN_ERR_STRIDE


def test_nulls_and_empty_batches():
    d = dims()
    for name in ("q", "k", "v", "pos", "inv_freq", "off", "ctx", "table", "qo", "kp", "vp", "status"):
        assert rope(d, **{name: None}) == G.GDN_ERR_NULL
    for name in ("q", "kp", "vp", "table", "ctx", "off", "o", "ws", "status"):
        assert attend(d, **{name: None}) == G.GDN_ERR_NULL
    for name in ("acc", "par", "off", "ctx", "table", "kp", "vp", "nl", "status"):
        assert move(d, **{name: None}) == G.GDN_ERR_NULL
    for name in ("p", "tok", "par", "off", "u", "un", "acc", "nt", "na", "status"):
        assert accept(**{name: None}) == G.GDN_ERR_NULL
    e = dims(n_seqs=0, n_tokens=0)
    assert rope(e, q=None) == attend(e, q=None) == move(e, acc=None) == G.GDN_OK
    assert accept(G.GdnDims.make(0, 0, 1, 1, 1, 16, 16), p=None) == G.GDN_OK
    assert rope(dims(n_tokens=0)) == attend(dims(n_tokens=0)) == move(d, layers=0) == G.GDN_OK


def test_rope_refusals():
    d = dims()
    for bad in (dict(rot=8), dict(rot=80), dict(rot=-16), dict(n_axes=0), dict(n_axes=5), dict(inter=2), dict(eps=-1.0),
                dict(eps=float("nan"))):
        assert rope(d, **bad) == G.GDN_ERR_ARG
    for bad in (dict(qs=d.h_q * 64 - 8), dict(qs=d.h_q * 64 + 4), dict(ks=64), dict(vs=d.h_kv * 64 + 1), dict(qos=0)):
        assert rope(d, **bad) == G.GDN_ERR_STRIDE
    for bad in (dict(q=FAKE + 8), dict(kp=13 * FAKE + 2), dict(qw=4 * FAKE + 4), dict(inv_freq=7 * FAKE + 4)):
        assert rope(d, **bad) == G.GDN_ERR_ALIGN
    for bad in (dict(qo=2 * FAKE), dict(kp=FAKE), dict(vp=12 * FAKE), dict(qo=FAKE + 16), dict(qo=FAKE, qos=d.h_q * 64 + 8)):
        assert rope(d, **bad) == G.GDN_ERR_ALIAS


def test_attention_refusals():
    d = dims()
    for s in (0.0, -1.0, float("nan"), float("inf")):
        assert attend(d, scale=s) == G.GDN_ERR_ARG
    assert attend(d, wb=G.gdn_attention_workspace_bytes(d) - 1) == G.GDN_ERR_ARG
    assert attend(d, wb=-1) == G.GDN_ERR_ARG
    assert attend(dims(max_seq_tokens=65), par=FAKE * 7) == G.GDN_ERR_DIMS
    assert attend(d, qs=d.h_q * 64 + 4) == G.GDN_ERR_STRIDE
    assert attend(d, o=8 * FAKE + 8) == G.GDN_ERR_ALIGN
    assert attend(d, o=FAKE) == attend(d, o=2 * FAKE + 64) == attend(d, ws=3 * FAKE) == G.GDN_ERR_ALIAS


def test_move_refusals():
    d = dims()
    assert move(dims(max_seq_tokens=65)) == G.GDN_ERR_DIMS
    assert move(d, layers=-1) == G.GDN_ERR_ARG
    assert move(d, ls=-8) == move(d, ls=12) == G.GDN_ERR_STRIDE
    assert move(d, kp=6 * FAKE + 8) == G.GDN_ERR_ALIGN
    assert move(d, nl=4 * FAKE) == move(d, kp=5 * FAKE) == G.GDN_ERR_ALIAS


def test_accept_refusals():
    assert accept(vocab=0) == accept(rep=2) == accept(vocab=1 << 29) == G.GDN_ERR_ARG
    assert accept(ps=96) == accept(ps=102) == accept(qs=98) == accept(vocab=101) == G.GDN_ERR_STRIDE
    assert accept(p=FAKE + 4) == accept(q=2 * FAKE + 8) == G.GDN_ERR_ALIGN
    assert accept(acc=4 * FAKE) == accept(nt=8 * FAKE) == accept(na=FAKE + 16) == G.GDN_ERR_ALIAS
    assert accept(G.GdnDims.make(2, 8, 1, 1, 1, 16, 65)) == G.GDN_ERR_DIMS


def test_reference_attention_of_equal_keys_is_the_mean():
    rng = np.random.default_rng(0)
    c = R.make_cache(rng, [5], 1, 64, 8, torch.bfloat16)
    for x in range(5):
        c.k[c.index(0, x)] = 1.0
    q = torch.randn(2, 2, 64, dtype=torch.float64)
    o, _, _ = R.attention(q, c, [3], [2], None, 0.125)
    v = c.view(c.v, 0, 5)[:, 0]
    assert torch.allclose(o[0, 0], v[:4].mean(0)) and torch.allclose(o[1, 1], v.mean(0))
    o, _, _ = R.attention(q, c, [3], [2], [[-1, -1]], 0.125)      # two roots: siblings do not see each other
    assert torch.allclose(o[1, 0], v[[0, 1, 2, 4]].mean(0))


def test_reference_rope_turns_by_the_angle():
    x = torch.zeros(1, 1, 64, dtype=torch.float64)
    x[..., 0] = 1.0
    z, _ = R.rope(x, np.array([[3]]), [0.5] * 8, [0] * 8, 16, False)
    assert math.isclose(z[0, 0, 0], math.cos(1.5)) and math.isclose(z[0, 0, 8], math.sin(1.5))
    z, _ = R.rope(x, np.array([[3]]), [0.5] * 8, [0] * 8, 16, True)
    assert math.isclose(z[0, 0, 1], math.sin(1.5))


@pytest.mark.parametrize("mode", ["without", "with", "none"])
def test_reference_acceptance_keeps_the_target_distribution(mode):
    """The first token that comes out (an accepted child's, or the next token) is
    distributed as p: 20,000 draws, within 5 standard deviations per token."""
    rng = np.random.default_rng(5)
    V, n = 5, 20000
    p, q = rng.dirichlet(np.ones(V)), rng.dirichlet(np.ones(V))
    got = np.zeros(V)
    for _ in range(n):
        kids = (rng.choice(V, 3, replace=mode == "with", p=q) if mode != "none" else np.array([1, 4, 0]))
        a, t, m = R.accept([-1, 0, 0, 0], [0, *kids], np.tile(p, (4, 1)), np.tile(q, (4, 1)) if mode != "none" else None,
                           rng.random(4), rng.random(), mode == "with")
        got[t if a == 0 else kids[a - 1]] += 1
    sd = np.sqrt(n * p * (1 - p))
    assert np.all(np.abs(got - n * p) <= 5 * sd)
