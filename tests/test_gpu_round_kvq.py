"""The 4-bit cache's operators and the sampling's as one round, as they are used:
rope into 16-bit rows -> append -> attention -> logits to probabilities of target and
draft -> acceptance -> commits of the cache and of the token history.  A captured graph
gives what the calls give, a tree round leaves the cache and the history that plain
decoding of the accepted tokens leaves, and greedy rounds accept what plain decoding
would have produced."""
import numpy as np
import pytest
import torch

import attn_ref as R
import gated_deltanet_speculative_gdn_gb300 as G
import kv4_ref as Q

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # collected on CPU machines, never run there
    pytest.skip("needs a CUDA GPU", allow_module_level=True)


def i32(x):
    return torch.tensor(np.asarray(x, dtype=np.int32), device="cuda")


class Round4:
    """S sequences whose draft proposes the same tree of tokens each round; the model's layers between the operators
    are random draws."""
    S, NODES, VOCAB, PAGE, PAGES_PER_SEQ, SLOTS = 4, 16, 1003, 16, 12, 6
    HQ, HKV, D, ROT = 8, 2, 128, 64
    PARENTS = [-1, 0, 0, 1, 1, 2, 2, 3, 3, 4, 5, 5, 7, 8, 10, 12]

    def __init__(self, seed):
        S, n = self.S, self.NODES
        N = S * n
        self.g = torch.Generator(device="cuda").manual_seed(seed)
        e = dict(device="cuda")
        self.dims = G.GdnDims.make(S, N, self.SLOTS, 1, 1, 128, n)
        self.adims = G.AttnDims.make_kvq(S, N, n, self.HQ, self.HKV, self.D, G.GDN_BF16, S * self.PAGES_PER_SEQ, self.PAGE, self.PAGES_PER_SEQ)
        # the new tokens' 16-bit rows, as pages of one sequence for the rotary step
        self.rdims = G.AttnDims.make(1, N, N, self.HQ, self.HKV, self.D, G.GDN_BF16, N // 8, 8, N // 8)
        self.one_off, self.zero, self.rows = i32([0, N]), i32([0]), torch.arange(N // 8, dtype=torch.int32, **e)
        self.kr, self.vr = (torch.zeros(N, self.HKV * self.D, dtype=torch.bfloat16, **e) for _ in range(2))
        shape = (S * self.PAGES_PER_SEQ, self.HKV, G.gdn_kvq_block_bytes(self.adims))
        self.k_pool, self.v_pool = (torch.zeros(shape, dtype=torch.uint8, **e) for _ in range(2))
        self.table = torch.randperm(S * self.PAGES_PER_SEQ, generator=self.g, **e).to(torch.int32).view(S, -1)
        self.ctx_len, self.new_len = (torch.zeros(S, dtype=torch.int32, **e) for _ in range(2))
        self.parents, self.node_off = i32(self.PARENTS * S), torch.arange(0, N + 1, n, dtype=torch.int32, **e)
        self.slot_map = i32([5, 0, 3, 2])
        self.depth = i32([len(R.path_of(self.PARENTS, i)) - 1 for i in range(n)] * S)
        self.pos = torch.zeros(N, 1, dtype=torch.int32, **e)
        half = self.ROT // 2
        self.inv_freq = torch.tensor([1e6 ** (-i / half) for i in range(half)], dtype=torch.float64, **e)
        self.q, self.qr, self.ao = (torch.zeros(N, self.HQ * self.D, dtype=torch.bfloat16, **e) for _ in range(3))
        self.k, self.v = (torch.zeros(N, self.HKV * self.D, dtype=torch.bfloat16, **e) for _ in range(2))
        self.work = torch.empty(G.gdn_attention_kvq_workspace_bytes(self.adims), dtype=torch.uint8, **e)
        self.P = (self.VOCAB + 7) // 8 * 8
        self.logits, self.draft = (torch.zeros(N, self.P, dtype=torch.bfloat16, **e) for _ in range(2))
        self.p, self.pd = (torch.zeros(N, self.P, **e) for _ in range(2))
        self.history = torch.zeros(self.SLOTS, self.P, dtype=torch.int16, **e)
        self.rep, self.freq, self.pres = (torch.full((S,), x, **e) for x in (1.2, 0.2, 0.1))
        self.temp = torch.tensor([0.9, 1.0, 0.7, 1.1], **e)
        self.mask = torch.full((2, (self.VOCAB + 31) // 32), 0x55555555, dtype=torch.int32, **e)
        self.mask_row = i32([0] * n + [-1] * n + [1] * n + [-1] * n)
        self.tokens = torch.zeros(N, dtype=torch.int32, **e)
        self.u, self.u_next = torch.zeros(N, **e), torch.zeros(S, **e)
        self.accepted, self.next_token, self.count = (torch.zeros(S, dtype=torch.int32, **e) for _ in range(3))
        self.status = torch.zeros(1, dtype=torch.int32, **e)

    def draw(self):
        for t in (self.q, self.k, self.v):
            t.copy_(torch.randn(t.shape, generator=self.g, device="cuda"))
        logits = torch.randn(self.logits.shape, generator=self.g, device="cuda") * 3
        self.logits.copy_(logits)
        self.draft.copy_(logits + 0.5 * torch.randn(logits.shape, generator=self.g, device="cuda"))
        self.tokens.copy_(2 * torch.randint(0, self.VOCAB // 2, self.tokens.shape, generator=self.g, device="cuda"))
        # children that the target likes, so that some are accepted
        best = self.draft[:, :self.VOCAB].float()
        best[:, 1::2] -= 100.0
        top = best.topk(3, dim=1).indices
        rank = [sum(1 for j in range(i) if self.PARENTS[j] == self.PARENTS[i]) for i in range(self.NODES)]
        for s in range(self.S):
            for i in range(1, self.NODES):
                self.tokens[s * self.NODES + i] = top[s * self.NODES + self.PARENTS[i], rank[i]].to(torch.int32)
        self.u.uniform_(generator=self.g)
        self.u_next.uniform_(generator=self.g)

    def probs(self, logits, p):
        G.gdn_logits_probs(self.dims, self.VOCAB, G.GDN_BF16, logits, self.P, self.tokens, self.parents, self.node_off, self.slot_map, self.history, self.P,
                           self.rep, self.freq, self.pres, self.temp, None, None, None, 0, self.mask, self.mask.stride(0), self.mask_row, 2, p, self.P,
                           self.status)

    def step(self):
        w, kw = self.HQ * self.D, self.HKV * self.D
        torch.add(self.ctx_len.repeat_interleave(self.NODES), self.depth, out=self.pos.view(-1))
        G.gdn_rope_append(self.rdims, self.q, w, self.k, kw, self.v, kw, None, None, 0.0, self.pos, 1, self.inv_freq, None, self.ROT, 0, self.one_off,
                          self.zero, self.rows, self.qr, w, self.kr, self.vr, self.status)
        G.gdn_kvq_append(self.adims, self.kr, kw, self.vr, kw, 1.0, 0.5, self.node_off, self.ctx_len, self.table, self.k_pool, self.v_pool, self.status)
        G.gdn_paged_attention_kvq(self.adims, self.qr, w, self.k_pool, self.v_pool, 1.0, 0.5, self.table, self.ctx_len, self.node_off, self.parents,
                                  self.D ** -0.5, self.ao, self.work, self.work.numel(), self.status)
        self.probs(self.logits, self.p)
        self.probs(self.draft, self.pd)
        G.gdn_tree_accept(self.dims, self.VOCAB, self.p, self.P, self.pd, self.P, 0, self.tokens, self.parents, self.node_off, self.u, self.u_next,
                          self.accepted, self.next_token, self.count, self.status)
        G.gdn_kvq_commit(self.adims, 1, 0, self.accepted, self.parents, self.node_off, self.ctx_len, self.table, self.k_pool, self.v_pool, self.new_len,
                         self.status)
        G.gdn_token_commit(self.dims, self.VOCAB, self.tokens, self.accepted, self.parents, self.node_off, self.slot_map, 0, self.history, self.P, self.status)
        self.ctx_len.copy_(self.new_len)


STATE = ("k_pool", "v_pool", "ctx_len", "accepted", "next_token", "count", "ao", "p", "pd", "history")


def test_graph_replay_equals_the_calls():
    a, b = Round4(3), Round4(3)
    a.draw(), b.draw()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b.step()
    taken = 0
    for _ in range(6):
        a.step()
        graph.replay()
        torch.cuda.synchronize()
        assert int(a.status) == int(b.status) == 0
        for name in STATE:
            assert bool(torch.equal(getattr(a, name), getattr(b, name))), name
        taken += int(a.count.sum())
        a.draw(), b.draw()
    assert taken > 6 * a.S                                        # something beyond the roots was accepted


def test_round_leaves_what_plain_decoding_leaves():
    """The accepted path's rows and counts are those of its tokens one by one, and its outputs agree."""
    r = Round4(7)
    for _ in range(3):
        r.draw()
        r.step()
    r.draw()
    d = Round4(7)
    for name in ("k_pool", "v_pool", "ctx_len", "history", "table"):
        setattr(d, name, getattr(r, name).clone())
    before = r.ctx_len.tolist()
    r.step()
    torch.cuda.synchronize()
    assert int(r.status) == 0
    S, n, kw = r.S, r.NODES, r.HKV * r.D
    paths = [R.path_of(r.PARENTS, a) for a in r.accepted.tolist()]
    for j in range(max(len(p) for p in paths)):
        live = [s for s in range(S) if j < len(paths[s])]
        at = torch.tensor([s * n + paths[s][j] for s in live], device="cuda")
        counts = [1 if s in live else 0 for s in range(S)]
        off = i32(np.concatenate([[0], np.cumsum(counts)]))
        lens = i32([before[s] + min(j, len(paths[s])) for s in range(S)])
        ad = G.AttnDims.make_kvq(S, len(live), 1, r.HQ, r.HKV, r.D, G.GDN_BF16, S * r.PAGES_PER_SEQ, r.PAGE, r.PAGES_PER_SEQ)
        G.gdn_kvq_append(ad, r.kr[at].contiguous(), kw, r.vr[at].contiguous(), kw, 1.0, 0.5, off, lens, d.table, d.k_pool, d.v_pool, d.status)
        o = torch.zeros(len(live), r.HQ * r.D, dtype=torch.bfloat16, device="cuda")
        G.gdn_paged_attention_kvq(ad, r.qr[at].contiguous(), r.HQ * r.D, d.k_pool, d.v_pool, 1.0, 0.5, d.table, lens, off, None, r.D ** -0.5, o, d.work,
                                  d.work.numel(), d.status)
        # |v| < 6: each call is within 2^-8 |o| (the result's rounding) + 2^-11 6 (the weights' in fp16) of the exact result,
        # and 2^-9 6 is more than what 32-bit scores move the weights by
        assert float((o.double() - r.ao[at].double()).abs().max()) <= 2 * (2.0 ** -8 + 2.0 ** -11 + 2.0 ** -9) * 6
        gd = G.GdnDims.make(S, len(live), r.SLOTS, 1, 1, 128, 1)
        G.gdn_token_commit(gd, r.VOCAB, r.tokens[at].contiguous(), None, None, off, r.slot_map, 0, d.history, r.P, d.status)
    torch.cuda.synchronize()
    assert int(d.status) == 0
    assert r.ctx_len.tolist() == [b + len(p) for b, p in zip(before, paths)]
    assert torch.equal(r.history, d.history)
    c = Q.Cache4(r.k_pool.view(-1).cpu(), r.v_pool.view(-1).cpu(), r.table.cpu().numpy(), r.PAGE, S * r.PAGES_PER_SEQ,
                 (r.adims.page_stride, r.adims.head_stride), r.HKV, r.D, (1.0, 0.5))
    for s in range(S):
        for x in range(before[s] + len(paths[s])):
            for mine, other in ((c.k, d.k_pool), (c.v, d.v_pool)):
                flat = other.view(-1).cpu()
                for ix in (c.codes_at(s, x), c.scales_at(s, x)):
                    assert torch.equal(mine[ix], flat[ix])


def test_prompt_then_rounds():
    """A prompt's tokens into the history and its rows into the cache, in chunks that end inside a page, then rounds on it:
    the penalties see the prompt."""
    r = Round4(11)
    new, kw = [37, 5, 64, 20], r.HKV * r.D
    N = sum(new)
    off = i32(np.concatenate([[0], np.cumsum(new)]))
    tokens = torch.randint(0, r.VOCAB, (N,), generator=r.g, device="cuda").to(torch.int32)
    G.gdn_token_commit(G.GdnDims.make(r.S, N, r.SLOTS, 1, 1, 128, 64), r.VOCAB, tokens, None, None, off, r.slot_map, 1, r.history, r.P, r.status)
    k, v = (torch.randn(N, kw, generator=r.g, device="cuda").bfloat16() for _ in range(2))
    ad = G.AttnDims.make_kvq(r.S, N, max(new), r.HQ, r.HKV, r.D, G.GDN_BF16, r.S * r.PAGES_PER_SEQ, r.PAGE, r.PAGES_PER_SEQ)
    G.gdn_kvq_append(ad, k, kw, v, kw, 1.0, 0.5, off, r.ctx_len, r.table, r.k_pool, r.v_pool, r.status)
    r.ctx_len.copy_(i32(new))
    h = r.history.cpu().numpy().view(np.uint16)
    for s in range(r.S):
        want = np.zeros(r.P, np.uint16)
        want[tokens[int(off[s]):int(off[s + 1])].cpu().numpy()] = 0x8000
        assert np.array_equal(h[int(r.slot_map[s])], want)
    for _ in range(3):
        r.draw()
        r.step()
    torch.cuda.synchronize()
    assert int(r.status) == 0
    assert all(int(c) > b for c, b in zip(r.ctx_len.tolist(), new))
    made = r.history.cpu().numpy().view(np.uint16).astype(int) & 0x7fff
    assert made.sum() == sum(r.ctx_len.tolist()) - N
