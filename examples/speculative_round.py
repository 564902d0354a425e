"""A speculative round of a small hybrid model's layer pair, on the device from draft to commit.

    python examples/speculative_round.py [rounds]

One GDN layer and one full-attention layer verify the same token trees; the
acceptance is decided on the device and both layers commit the accepted path:

    gdn_conv_tree_step_compact -> gdn_tree_verify        (GDN layer)
    gdn_rope_append -> gdn_paged_attention               (attention layer)
    gdn_tree_accept                                      (accepted nodes, next tokens)
    gdn_commit_compact, gdn_kv_commit                    (both layers' state)

No step waits for the host, so the round is captured into one CUDA graph and
replayed; between replays the host only draws new inputs.  Weights, activations
and distributions are random: it shows the calls, not a language model.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import gated_deltanet_speculative_gdn_gb300 as G  # noqa: E402


class Round:
    """The tensors of a batch of S sequences and one call per step of the round."""

    S, NODES, VOCAB, PAGE, PAGES_PER_SEQ = 4, 16, 1000, 32, 8
    HK, HV, D = 2, 4, 128            # GDN layer
    HQ, HKV, DH, ROT = 8, 2, 128, 64  # attention layer
    PARENTS = [-1, 0, 0, 1, 1, 2, 2, 3, 3, 4, 5, 5, 7, 8, 10, 12]

    def __init__(self, seed=0):
        S, n, dev = self.S, self.NODES, "cuda"
        N = S * n
        self.g = torch.Generator(device=dev).manual_seed(seed)
        self.dims = G.GdnDims.make(S, N, S, self.HK, self.HV, self.D, n)
        self.C = C = self.dims.conv_channels
        self.rs = G.gdn_replay_row_floats(self.D, self.D)
        self.adims = G.AttnDims.make(S, N, n, self.HQ, self.HKV, self.DH, G.GDN_BF16, S * self.PAGES_PER_SEQ, self.PAGE,
                                     self.PAGES_PER_SEQ)

        def f32(*shape, std=1.0):
            return torch.randn(shape, generator=self.g, device=dev) * std

        def empty(*shape, dtype=torch.float32):
            return torch.empty(shape, dtype=dtype, device=dev)

        i32 = dict(dtype=torch.int32, device=dev)
        self.parents = torch.tensor(self.PARENTS * S, **i32)
        self.node_off = torch.arange(0, N + 1, n, **i32)
        self.slot_map = torch.arange(S, **i32)
        self.depth = torch.tensor([self._depth(i) for i in range(n)] * S, **i32)
        self.status = torch.zeros(1, **i32)
        # GDN layer: weights, state, outputs
        self.conv_w, self.dt_bias, self.A = f32(C, 4, std=0.25), f32(self.HV), -f32(self.HV).abs() - 0.1
        self.ssm, self.hist = f32(S, self.HV, self.D, self.D, std=0.1), f32(S, 3, C)
        self.x, self.ba = empty(N, C), empty(N, 2 * self.HV)
        self.xc, self.win_ref = empty(N, C), empty(N, 3, dtype=torch.int32)
        self.o, self.replay = empty(N, self.HV, self.D), empty(N, self.HV, self.rs)
        # attention layer: cache, lengths, outputs
        shape = (S * self.PAGES_PER_SEQ, self.PAGE, self.HKV, self.DH)
        self.k_pool, self.v_pool = (torch.zeros(shape, dtype=torch.bfloat16, device=dev) for _ in range(2))
        self.table = torch.randperm(S * self.PAGES_PER_SEQ, generator=self.g, device=dev).to(torch.int32).view(S, -1)
        self.ctx_len, self.new_len = torch.zeros(S, **i32), torch.zeros(S, **i32)
        self.q, self.qr = (empty(N, self.HQ * self.DH, dtype=torch.bfloat16) for _ in range(2))
        self.k, self.v = (empty(N, self.HKV * self.DH, dtype=torch.bfloat16) for _ in range(2))
        self.q_norm, self.k_norm = 1 + f32(self.DH, std=0.1), 1 + f32(self.DH, std=0.1)
        half = self.ROT // 2
        self.inv_freq = torch.tensor([1e6 ** (-i / half) for i in range(half)], dtype=torch.float64, device=dev)
        self.pos = torch.zeros(N, 1, **i32)
        self.ao = empty(N, self.HQ * self.DH, dtype=torch.bfloat16)
        self.work = empty(G.gdn_attention_workspace_bytes(self.adims), dtype=torch.uint8)
        # acceptance
        self.p, self.qd = empty(N, self.VOCAB), empty(N, self.VOCAB)
        self.tokens = torch.zeros(N, **i32)
        self.u, self.u_next = empty(N), empty(S)
        self.accepted, self.next_token, self.count = (torch.zeros(S, **i32) for _ in range(3))

    def _depth(self, i):
        return 0 if i == 0 else 1 + self._depth(self.PARENTS[i])

    def draw(self):
        """New projections, distributions and uniforms: what the rest of a model would compute."""
        for t in (self.x, self.ba):
            t.normal_(generator=self.g)
        for t in (self.q, self.k, self.v):
            t.copy_(torch.randn(t.shape, generator=self.g, device="cuda"))
        logits = torch.randn(self.p.shape, generator=self.g, device="cuda") * 3
        draft = logits + torch.randn(self.p.shape, generator=self.g, device="cuda")
        self.p.copy_(torch.softmax(logits, 1))
        self.qd.copy_(torch.softmax(draft, 1))
        # a node's children are distinct draws from the draft at that node
        best = (draft - torch.log(-torch.log(torch.rand(draft.shape, generator=self.g, device="cuda") * 0.999 + 5e-4))).topk(3, 1).indices
        rank = [sum(1 for j in range(i) if self.PARENTS[j] == self.PARENTS[i]) for i in range(self.NODES)]
        row = torch.arange(self.S, device="cuda")[:, None] * self.NODES + torch.tensor([max(p, 0) for p in self.PARENTS], device="cuda")
        self.tokens.copy_(best[row.view(-1), torch.tensor(rank * self.S, device="cuda")])
        self.u.uniform_(generator=self.g)
        self.u_next.uniform_(generator=self.g)

    def step(self):
        """The round: nine kernels' worth of calls, none of which waits for the host."""
        st, d, ad = self.status, self.dims, self.adims
        torch.add(self.ctx_len.repeat_interleave(self.NODES), self.depth, out=self.pos.view(-1))
        G.gdn_conv_tree_step_compact(d, self.x, self.C, self.conv_w, self.hist, self.parents, self.node_off, self.slot_map,
                                     self.xc, self.win_ref, st)
        G.gdn_tree_verify(d, self.xc, self.ba, 2 * self.HV, self.dt_bias, self.A, self.ssm, 1.0, self.parents, self.node_off,
                          self.slot_map, self.o, self.replay, self.rs, st)
        w, kw = self.HQ * self.DH, self.HKV * self.DH
        G.gdn_rope_append(ad, self.q, w, self.k, kw, self.v, kw, self.q_norm, self.k_norm, 1e-6, self.pos, 1, self.inv_freq,
                          None, self.ROT, 0, self.node_off, self.ctx_len, self.table, self.qr, w, self.k_pool, self.v_pool, st)
        G.gdn_paged_attention(ad, self.qr, w, self.k_pool, self.v_pool, self.table, self.ctx_len, self.node_off, self.parents,
                              self.DH ** -0.5, self.ao, self.work, self.work.numel(), st)
        G.gdn_tree_accept(d, self.VOCAB, self.p, self.VOCAB, self.qd, self.VOCAB, 0, self.tokens, self.parents, self.node_off,
                          self.u, self.u_next, self.accepted, self.next_token, self.count, st)
        G.gdn_commit_compact(d, self.accepted, self.parents, self.node_off, self.slot_map, self.replay, self.rs, self.x, self.C,
                             self.win_ref, self.ssm, self.hist, st)
        G.gdn_kv_commit(ad, 1, 0, self.accepted, self.parents, self.node_off, self.ctx_len, self.table, self.k_pool, self.v_pool,
                        self.new_len, st)
        self.ctx_len.copy_(self.new_len)

    def capture(self):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            self.step()
        return graph


def main(rounds=8):
    r = Round()
    r.draw()
    graph = r.capture()          # (capturing runs nothing)
    for i in range(rounds):
        r.draw()
        graph.replay()
        assert int(r.status) == 0, G.gdn_status_str(int(r.status))
        print(f"round {i}: accepted {r.count.tolist()} nodes, next tokens {r.next_token.tolist()}, "
              f"lengths {r.ctx_len.tolist()}")
    return r


if __name__ == "__main__":
    main(int(sys.argv[1]) if len(sys.argv) > 1 else 8)
