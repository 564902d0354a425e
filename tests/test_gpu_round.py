"""The attention layer's operators, the acceptance and both commits as one round:
a captured graph gives what the calls give, a tree round gives what plain decoding
of the accepted tokens gives, and the acceptance feeds both commits on the device."""
import numpy as np
import pytest
import torch

import attn_ref as R
import gated_deltanet_speculative_gdn_gb300 as G
from examples.speculative_round import Round

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # collected on CPU machines, never run there
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

STATE = ("ssm", "hist", "k_pool", "v_pool", "ctx_len", "accepted", "next_token", "count", "ao", "o")


def test_graph_replay_equals_the_calls():
    a, b = Round(3), Round(3)
    a.draw(), b.draw()
    graph = b.capture()
    for _ in range(5):
        a.step()
        graph.replay()
        torch.cuda.synchronize()
        assert int(a.status) == int(b.status) == 0
        for name in STATE:
            assert bool(torch.equal(getattr(a, name), getattr(b, name))), name
        a.draw(), b.draw()
    assert int(a.ctx_len.min()) >= 5


def test_acceptance_feeds_the_commits():
    """What the round commits is what the host would commit from the downloaded acceptance."""
    a, b = Round(5), Round(5)
    for r in (a, b):
        r.draw()
    a.step()
    torch.cuda.synchronize()
    # the same round with the acceptance taken through the host
    before = b.ctx_len.clone()
    accept = G.gdn_tree_accept
    try:
        def through_host(*args, **kw):
            rc = accept(*args, **kw)
            got = [b.accepted.cpu().numpy().copy(), b.next_token.cpu().numpy().copy(), b.count.cpu().numpy().copy()]
            for s in range(b.S):
                rows = slice(s * b.NODES, (s + 1) * b.NODES)
                want = R.accept(b.PARENTS, b.tokens[rows].cpu().numpy(), b.p[rows].cpu().numpy(), b.qd[rows].cpu().numpy(),
                                b.u[rows].cpu().numpy(), float(b.u_next[s]), False)
                assert want == tuple(int(x[s]) for x in got)
            b.accepted.copy_(torch.from_numpy(got[0]))
            return rc
        G.gdn_tree_accept = through_host
        b.step()
    finally:
        G.gdn_tree_accept = accept
    torch.cuda.synchronize()
    for name in STATE:
        assert bool(torch.equal(getattr(a, name), getattr(b, name))), name
    assert torch.equal(b.ctx_len, before + b.count)


@pytest.mark.parametrize("name,d,hq,hkv,page", [("bf16", 256, 16, 2, 16), ("fp16", 128, 8, 4, 8), ("bf16", 64, 6, 2, 32)])
def test_tree_round_equals_plain_decoding(name, d, hq, hkv, page):
    """Append, attend and commit of a tree leave the cache that appending the accepted
    path's tokens one by one leaves, bit for bit, and the path's outputs agree with the
    single-token outputs within the two calls' rounding."""
    dtype = R.DTYPES[name]
    rng = np.random.default_rng(d)
    ctx, n = [37, 5, 64], 12
    S, N = len(ctx), 12 * 3
    par = [R.random_tree(rng, n) for _ in ctx]
    acc = [max(range(n), key=lambda i, p=p: len(R.path_of(p, i))) for p in par]
    cache = R.make_cache(rng, [c + n for c in ctx], hkv, d, page, dtype, garbage=0.0)
    g = torch.Generator().manual_seed(2)
    q, k, v = ((torch.randn((N, h * d), generator=g)).to(dtype).cuda() for h in (hq, hkv, hkv))
    half = d // 4
    inv_freq = torch.tensor([1e4 ** (-i / half) for i in range(half)], dtype=torch.float64, device="cuda")
    i32 = lambda x: torch.tensor(np.asarray(x, dtype=np.int32), device="cuda")
    table, status = i32(cache.table), torch.zeros(1, dtype=torch.int32, device="cuda")
    code = G.GDN_BF16 if name == "bf16" else G.GDN_FP16

    def forward(kp, vp, rows, counts, lens, parents, pos):
        dm = G.AttnDims.make(S, sum(counts), max(counts), hq, hkv, d, code, cache.n_pages, page, cache.table.shape[1], *cache.strides)
        off = i32(np.concatenate([[0], np.cumsum(counts)]))
        qs, ks, vs = (t[rows].contiguous() for t in (q, k, v))
        qr, o = torch.empty_like(qs), torch.empty_like(qs)
        G.gdn_rope_append(dm, qs, hq * d, ks, hkv * d, vs, hkv * d, None, None, 0.0, i32(pos).view(-1, 1), 1, inv_freq, None,
                          2 * half, 0, off, i32(lens), table, qr, hq * d, kp, vp, status)
        ws = torch.empty(G.gdn_attention_workspace_bytes(dm), dtype=torch.uint8, device="cuda")
        G.gdn_paged_attention(dm, qr, hq * d, kp, vp, table, i32(lens), off, None if parents is None else i32(parents),
                              d ** -0.5, o, ws, ws.numel(), status)
        return dm, off, o

    kt, vt = cache.k.cuda(), cache.v.cuda()
    rows = torch.arange(N, device="cuda")
    pos = [ctx[s] + len(R.path_of(par[s], i)) - 1 for s in range(S) for i in range(n)]
    dm, off, tree_o = forward(kt, vt, rows, [n] * S, ctx, [x for p in par for x in p], pos)
    new_len = torch.zeros(S, dtype=torch.int32, device="cuda")
    G.gdn_kv_commit(dm, 1, 0, i32(acc), i32([x for p in par for x in p]), off, i32(ctx), table, kt, vt, new_len, status)

    kd, vd = cache.k.cuda(), cache.v.cuda()
    paths = [R.path_of(par[s], acc[s]) for s in range(S)]
    h = R.half_step(dtype)
    for j in range(max(len(p) for p in paths)):
        live = [s for s in range(S) if j < len(paths[s])]
        counts = [1 if s in live else 0 for s in range(S)]
        at = torch.tensor([s * n + paths[s][j] for s in live], device="cuda")
        _, _, o = forward(kd, vd, at, counts, [ctx[s] + min(j, len(paths[s])) for s in range(S)], None, [ctx[s] + j for s in live])
        torch.cuda.synchronize()
        # |v| < 6 in these draws, so each call is within h |o| + (h + 2^-9) 6 of the exact result
        assert float((o.double() - tree_o[at].double()).abs().max()) <= 2 * (2 * h + 2.0 ** -9) * 6
    assert int(status) == 0
    assert new_len.tolist() == [ctx[s] + len(paths[s]) for s in range(S)]
    for s in range(S):
        for x in range(ctx[s] + len(paths[s])):
            ix = cache.index(s, x).cuda()
            assert torch.equal(kt[ix], kd[ix]) and torch.equal(vt[ix], vd[ix])
