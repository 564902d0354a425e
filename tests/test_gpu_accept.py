"""Acceptance of drafted trees on the GPU against the definition in 64 bits: whole
numbers, equal.  (Decisions closer than 2^-40 to a border could differ; the inputs
are random, so none is.)"""
import numpy as np
import pytest
import torch

import attn_ref as R
import gated_deltanet_speculative_gdn_gb300 as G

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # collected on CPU machines, never run there
    pytest.skip("needs a CUDA GPU", allow_module_level=True)


def run(par, tok, p, q, u, un, V, rep, max_nodes=None, off=None, S=None):
    new = [len(x) for x in par]
    S, N = len(new), sum(new)
    off = np.concatenate([[0], np.cumsum(new)]) if off is None else off
    dm = G.GdnDims.make(S, N, 1, 1, 1, 16, max_nodes or max(1, *new))
    t = lambda a, ty=torch.int32: torch.tensor(np.concatenate(a) if N else np.zeros(1), device="cuda").to(ty)
    out = [torch.full((S,), -9, dtype=torch.int32, device="cuda") for _ in range(3)]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    pd = torch.tensor(p, device="cuda")
    qd = None if q is None else torch.tensor(q, device="cuda")
    G.gdn_tree_accept(dm, V, pd, pd.stride(0), qd, 0 if q is None else qd.stride(0), rep, t(tok), t(par),
                      torch.tensor(off, dtype=torch.int32, device="cuda"), t(u, torch.float32),
                      torch.tensor(np.asarray(un, dtype=np.float32), device="cuda"), *out, status)
    torch.cuda.synchronize()
    return [x.cpu().tolist() for x in out], int(status)


def draw(seed, sizes, V, mode, kind="tree", std=2.0, noise=1.0, pad=float("nan")):
    rng = np.random.default_rng(seed)
    par, tok, u, ps, qs = [], [], [], [], []
    width = (V + 3) // 4 * 4 + 4
    for n in sizes:
        tree = R.random_tree(rng, n) if kind == "tree" else [i - 1 for i in range(n)] if kind == "chain" else [-1] + [0] * (n - 1)
        tree = tree[:n]
        x = rng.normal(size=(n, V)) * std
        y = x + rng.normal(size=(n, V)) * noise
        P, Q = (np.full((n, width), pad, np.float32) for _ in range(2))
        for z, to in ((x, P), (y, Q)):
            e = np.exp(z - z.max(1, keepdims=True))
            to[:, :V] = e / e.sum(1, keepdims=True)
        t = np.full(n, -5)
        for node in range(n):
            kids = [c for c in range(n) if tree[c] == node]
            if not kids:
                continue
            if mode == "none":
                t[kids] = np.argsort(-y[node])[np.arange(len(kids)) % V]
            elif mode == "with":
                t[kids] = rng.choice(V, len(kids), p=Q[node, :V].astype(np.float64) / Q[node, :V].astype(np.float64).sum())
            else:
                t[kids] = np.argsort(-(np.log(Q[node, :V].astype(np.float64)) + rng.gumbel(size=V)))[np.arange(len(kids)) % V]
        par.append(np.array(tree, dtype=np.int64))
        tok.append(t)
        u.append(rng.random(n).astype(np.float32))
        ps.append(P)
        qs.append(Q)
    p = np.concatenate(ps) if sum(sizes) else np.zeros((1, width), np.float32)
    q = None if mode == "none" else np.concatenate(qs) if sum(sizes) else np.zeros((1, width), np.float32)
    return par, tok, p, q, u, rng.random(len(sizes)).astype(np.float32)


def expect(par, tok, p, q, u, un, V, rep):
    out, at = [[], [], []], 0
    for s, tree in enumerate(par):
        n = len(tree)
        got = R.accept(list(tree), tok[s], p[at:at + n, :V], None if q is None else q[at:at + n, :V], u[s], un[s], rep)
        for k in range(3):
            out[k].append(got[k])
        at += n
    return out


@pytest.mark.parametrize("mode", ["without", "with", "none"])
@pytest.mark.parametrize("V,kind", [(1, "chain"), (2, "tree"), (3, "star"), (7, "tree"), (127, "tree"), (2050, "chain"),
                                    (4096, "star"), (32003, "tree")])
def test_accept(mode, V, kind):
    rng = np.random.default_rng(V)
    sizes = [int(x) for x in rng.integers(1, 17, 24)] + [0, 1, 2, 40 if V < 5000 else 8, 64 if V < 5000 else 9]
    a = draw(V, sizes, V, mode, kind)
    got, status = run(*a, V, int(mode == "with"))
    assert status == 0
    assert got == expect(*a, V, mode == "with")


@pytest.mark.parametrize("mode", ["without", "none"])
def test_accept_wide(mode):
    """The clusters' full width, flat rows (close borders) and peaked ones."""
    V = 131075
    for seed, std in ((1, 0.3), (2, 5.0)):
        a = draw(seed, [6, 1, 12, 3], V, mode, "tree", std=std)
        got, status = run(*a, V, 0)
        assert status == 0 and got == expect(*a, V, False)


def test_accept_identical_distributions_take_the_first_child():
    a = draw(3, [5] * 8, 500, "without", "chain", noise=0.0)
    got, status = run(*a, 500, 0)
    assert status == 0 and got[0] == [4] * 8 and got[2] == [5] * 8


def test_accept_greedy_target():
    """A one-hot target accepts its own token alone and answers with it otherwise."""
    V = 300
    par = [np.array([-1, 0, 0, 1])] * 3
    p = np.zeros((12, 304), np.float32)
    p[:, 17] = 1.0
    tok = [np.array([0, 17, 5, 17]), np.array([0, 5, 17, 3]), np.array([0, 5, 6, 17])]
    u = [np.full(4, 0.999, np.float32)] * 3
    got, status = run(par, tok, p, None, u, [0.5, 0.0, 0.999], V, 0)
    assert status == 0 and got == [[3, 2, 0], [17, 17, 17], [3, 2, 1]]


def test_accept_borders_of_the_uniforms():
    """u_next at 0, just under 1 and above: the first and the last token with mass."""
    V = 5000
    p = np.zeros((4, 5000), np.float32)
    p[:, 3:4000] = 1.0 / 3997
    got, status = run([np.array([-1])] * 4, [np.zeros(1, int)] * 4, p, None, [np.zeros(1, np.float32)] * 4,
                      [0.0, np.nextafter(np.float32(1), np.float32(0)), 1.0, -1.0], V, 0)
    assert status == 0
    assert got[1][0] == 3 and got[1][1] == 3999 and got[1][2] == 3999 and got[1][3] == 3


def test_accept_rows_without_meaning_stay_in_range():
    V = 1003
    for bad in (0.0, float("nan"), float("inf"), -1.0):
        p = np.full((6, 1004), bad, np.float32)
        for q in (None, p.copy()):
            got, status = run([np.array([-1, 0, 0])] * 2, [np.array([0, 1, 2])] * 2, p, q, [np.full(3, 0.5, np.float32)] * 2,
                              [0.3, 0.9], V, 0)
            assert status == 0 and all(0 <= x < V for x in got[1]) and all(0 <= x < 3 for x in got[0])


@pytest.mark.parametrize("what,code", [("root", G.GDN_DEV_BAD_PARENT), ("order", G.GDN_DEV_BAD_PARENT),
                                       ("two roots", G.GDN_DEV_BAD_PARENT), ("token", G.GDN_DEV_BAD_TOKEN),
                                       ("off", G.GDN_DEV_BAD_NODE_OFF), ("many", G.GDN_DEV_BAD_NODE_OFF)])
def test_accept_device_errors(what, code):
    par, tok, p, q, u, un = draw(4, [5, 5], 40, "without", "chain")
    kw = {}
    if what == "root":
        par[1][0] = 0
    elif what == "order":
        par[1][2] = 3
    elif what == "two roots":
        par[1][3] = -1
    elif what == "token":
        tok[1][3] = 40
    elif what == "off":
        kw["off"] = [0, 11, 10]
    else:
        kw["max_nodes"] = 4
    got, status = run(par, tok, p, q, u, un, 40, 0, **kw)
    assert status == code
    assert got[0][1] == -1 and got[1][1] == -1 and got[2][1] == 0


def test_accept_tokens_are_the_targets():
    """40,000 sequences of one tree: the first token that comes out follows p within
    5 standard deviations."""
    V, n = 6, 40000
    rng = np.random.default_rng(11)
    p1, q1 = (rng.dirichlet(np.ones(V)).astype(np.float32) for _ in range(2))
    width = 8
    p, q = (np.zeros((4 * n, width), np.float32) for _ in range(2))
    p[:, :V], q[:, :V] = p1, q1
    keys = np.log(q1.astype(np.float64)) + rng.gumbel(size=(n, V))
    kids = np.argsort(-keys, axis=1)[:, :3]
    par = [np.array([-1, 0, 0, 0])] * n
    tok = [np.array([0, *k]) for k in kids]
    u = list(rng.random((n, 4)).astype(np.float32))
    got, status = run(par, tok, p, q, u, rng.random(n).astype(np.float32), V, 0)
    assert status == 0
    first = [got[1][s] if got[0][s] == 0 else kids[s][got[0][s] - 1] for s in range(n)]
    count = np.bincount(first, minlength=V)
    sd = np.sqrt(n * p1.astype(np.float64) * (1 - p1))
    assert np.all(np.abs(count - n * p1.astype(np.float64)) <= 5 * sd)
