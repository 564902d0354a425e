"""Measured cases of the attention-layer and acceptance operators of a speculative round.

Four operators around one paged key/value cache:

  append   q/k RMS norm and rotary positions with several axes, then the new tokens' keys and values into the cache
  attend   attention of a chunk of new tokens (a prompt chunk, a token tree, one token) over the paged cache
  move     the accepted path's keys and values to their final places in the cache, for every layer at once
  accept   drafted token trees against the target's probabilities, from given random numbers

`own = False` computes them in elementary torch operations; `own = True` calls the library's entry points.
Lengths, trees and accepted nodes follow from the case; values, tokens and the page order from the seed.
"""
import math
import random

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


# ---- cases ------------------------------------------------------------------------------------------------------------------


def listed():
    return [
        # one user, one token: the smallest call, where latency counts
        {"name": "attend_one_token", "op": "attend", "type": "bf16", "seqs": 1, "new": 1, "ragged": False, "tree": False, "ctx": 777, "hq": 16, "hkv": 2,
         "d": 256, "page": 16},
        # a full batch of plain decode steps over contexts of very different lengths
        {"name": "attend_decode_batch", "op": "attend", "type": "bf16", "seqs": 64, "new": 1, "ragged": False, "tree": False, "ctx": 16384, "hq": 16, "hkv": 2,
         "d": 256, "page": 64},
        # the headline round: 64 sequences of 16-node trees, here in the full-attention layer
        {"name": "attend_trees", "op": "attend", "type": "bf16", "seqs": 64, "new": 16, "ragged": False, "tree": True, "ctx": 8192, "hq": 16, "hkv": 2,
         "d": 256, "page": 32},
        # a chunk of a long prompt
        {"name": "attend_prompt_chunk", "op": "attend", "type": "bf16", "seqs": 1, "new": 4096, "ragged": False, "tree": False, "ctx": 12288, "hq": 16,
         "hkv": 2, "d": 256, "page": 64},
        # chunks of several prompts in one call, odd lengths, the other type and head width
        {"name": "attend_mixed_chunks", "op": "attend", "type": "fp16", "seqs": 9, "new": 701, "ragged": True, "tree": False, "ctx": 3001, "hq": 32, "hkv": 8,
         "d": 128, "page": 16},
        # a round's few new tokens
        {"name": "append_trees", "op": "append", "type": "bf16", "seqs": 4, "new": 16, "ragged": False, "tree": True, "ctx": 1000, "hq": 16, "hkv": 2, "d": 256,
         "page": 32, "rot": 64, "axes": 1, "norm": True},
        # a prompt of image and text tokens, with three axes
        {"name": "append_prompt", "op": "append", "type": "bf16", "seqs": 3, "new": 4001, "ragged": True, "tree": False, "ctx": 50, "hq": 16, "hkv": 2, "d": 256,
         "page": 64, "rot": 64, "axes": 3, "norm": True},
        # one layer, few sequences; and all the attention layers of a stack for the headline batch
        {"name": "move_one_layer", "op": "move", "type": "bf16", "seqs": 4, "new": 16, "tree": True, "ctx": 500, "hkv": 2, "d": 256, "page": 16, "layers": 1},
        {"name": "move_stack", "op": "move", "type": "bf16", "seqs": 64, "new": 16, "tree": True, "ctx": 500, "hkv": 2, "d": 256, "page": 32, "layers": 12},
        # one user's tree; the headline batch; a batch of chains from a draft that proposes one token outright
        {"name": "accept_one_tree", "op": "accept", "seqs": 1, "new": 16, "ragged": False, "tree": True, "vocab": 131072, "draft": "without"},
        {"name": "accept_trees", "op": "accept", "seqs": 64, "new": 16, "ragged": False, "tree": True, "vocab": 131072, "draft": "without"},
        {"name": "accept_chains", "op": "accept", "seqs": 17, "new": 8, "ragged": True, "tree": False, "vocab": 50003, "draft": "none"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attend", "attend", "append", "move", "accept"])
    if op == "accept":
        tree = rng.random() < 0.7
        return {"op": op, "seqs": _log(rng, 1, 64), "new": rng.randint(2, 16), "ragged": rng.random() < 0.5, "tree": tree, "vocab": _log(rng, 1000, 131072),
                "draft": rng.choice(["without", "with", "none"])}
    d, hkv, group = rng.choice([(256, 2, 8), (256, 4, 4), (256, 2, 6), (128, 8, 4), (128, 4, 5), (64, 8, 1)])
    c = {"op": op, "type": rng.choice(["bf16", "fp16"]), "hkv": hkv, "d": d, "page": rng.choice([16, 32, 64, 128])}
    if op == "move":
        return {**c, "seqs": _log(rng, 1, 64), "new": rng.randint(2, 32), "tree": rng.random() < 0.7, "ctx": _log(rng, 1, 500), "layers": rng.randint(1, 12)}
    c["hq"] = hkv * group
    kind = rng.choice(["decode", "tree", "chunk"])
    if kind == "decode":
        c |= {"seqs": _log(rng, 1, 64), "new": 1, "ragged": False, "tree": False, "ctx": _log(rng, 1, 12000)}
    elif kind == "tree":
        c |= {"seqs": _log(rng, 1, 48), "new": rng.randint(2, 40), "ragged": rng.random() < 0.5, "tree": True, "ctx": _log(rng, 1, 5000)}
    else:
        c |= {"seqs": rng.randint(1, 5), "new": _log(rng, 17, 1200), "ragged": True, "tree": False, "ctx": _log(rng, 1, 4000)}
    if op == "append":
        c |= {"rot": rng.choice([d // 4, d // 2, d]), "axes": rng.choice([1, 3]), "norm": rng.random() < 0.5}
    return c


# ---- structure: lengths, trees, accepted nodes (from the case alone) --------------------------------------------------------------


def _parents(n, tree, r):
    if not tree:
        return [i - 1 for i in range(n)]
    par, depth, kids = [-1], [1], [0]
    for i in range(1, n):
        p = r.choice([j for j in range(i) if depth[j] < 8 and kids[j] < 3] or [i - 1])
        par.append(p)
        depth.append(depth[p] + 1)
        kids.append(0)
        kids[p] += 1
    return par


def _structure(c):
    r = random.Random(1000 * c["seqs"] + c["new"])
    S, n = c["seqs"], c["new"]
    new = [max(1, n - (i * n) // (2 * S)) if c.get("ragged") else n for i in range(S)]
    ctx = [max(1, int(c.get("ctx", 0) * (1 - 0.9 * ((i * 0.6180339887) % 1.0)))) for i in range(S)]
    par = [_parents(k, c["tree"], r) for k in new] if n <= 64 else None
    acc = [r.randrange(k) for k in new] if par else None
    return new, ctx, par, acc


def _path(par, node):
    p = []
    while node >= 0:
        p.append(node)
        node = par[node]
    return p[::-1]


def work(c):
    new, ctx, par, acc = _structure(c)
    N = sum(new)
    if c["op"] == "accept":
        # at least the row that the next token comes from; with draft probabilities the draft's row too (a walk that ends in a rejection)
        return {"bytes": c["seqs"] * c["vocab"] * 4 * (1 if c["draft"] == "none" else 2) + 16 * N, "flops": c["seqs"] * c["vocab"] * (1 if c["draft"] == "none" else 4)}
    row = 2 * c["d"]
    if c["op"] == "move":
        moved = sum(1 for p, a in zip(par, acc) for j, x in enumerate(_path(p, a)) if x != j)
        return {"bytes": moved * 2 * 2 * c["hkv"] * row * c["layers"] + 8 * N, "flops": 0}
    rows = c["hq"] + 2 * c["hkv"]
    if c["op"] == "append":
        return {"bytes": 2 * N * rows * row + 4 * N * c["axes"], "flops": N * (c["hq"] + c["hkv"]) * (3 * c["rot"] + (3 * c["d"] if c["norm"] else 0))}
    seen = [sum(ctx[s] + (len(_path(par[s], i)) if c["tree"] else i + 1) for i in range(new[s])) for s in range(c["seqs"])]
    return {"bytes": sum((a + b) for a, b in zip(ctx, new)) * 2 * c["hkv"] * row + 2 * N * c["hq"] * row, "flops": 4 * c["d"] * c["hq"] * sum(seen)}


# ---- inputs -----------------------------------------------------------------------------------------------------------------------


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def prepare(c, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, std=1.0, dtype=torch.float32):
        return torch.randn(shape, generator=g, device="cuda", dtype=dtype).mul_(std)

    new, ctx, par, acc = _structure(c)
    S, N = c["seqs"], sum(new)
    off = [0]
    for k in new:
        off.append(off[-1] + k)
    s = {"case": c, "node_off": _i32(off), "off": off, "new": new, "status": torch.zeros(1, dtype=torch.int32, device="cuda"),
         "parents": _i32([x for p in par for x in p]) if c["tree"] or c["op"] in ("move", "accept") else None}
    if own:
        import gated_deltanet_speculative_gdn_gb300 as G
        s["G"] = G
    if c["op"] == "accept":
        V, P = c["vocab"], (c["vocab"] + 3) // 4 * 4
        logits = normal(N, V, std=3.0)
        p = torch.zeros(N, P, device="cuda")
        p[:, :V] = torch.softmax(logits, dim=1)
        q, scores = None, logits
        if c["draft"] != "none":  # the draft: the target's logits with noise
            logits += normal(N, V, std=1.0)
            q = torch.zeros(N, P, device="cuda")
            q[:, :V] = torch.softmax(logits, dim=1)
            # children drawn from the draft without replacement: the k largest of log q + Gumbel noise
            scores = logits - torch.log(-torch.log(torch.rand(N, V, generator=g, device="cuda").clamp_(1e-30, 1 - 1e-7)))
        top = scores.topk(3, dim=1).indices
        kids, parent_row, rank = {}, [], []
        for k in range(S):
            for i, x in enumerate(par[k]):
                parent_row.append(off[k] + max(x, 0))
                rank.append(kids.get((k, x), 0) if x >= 0 else 0)
                kids[(k, x)] = kids.get((k, x), 0) + 1
        tokens = top[torch.tensor(parent_row, device="cuda"), torch.tensor(rank, device="cuda")].to(torch.int32)
        if c["draft"] == "with":  # with replacement: independent draws
            again = torch.multinomial(q[:, :V], 3, replacement=True, generator=g)
            tokens = again[torch.tensor(parent_row, device="cuda"), torch.tensor(rank, device="cuda")].to(torch.int32)
        s |= {"p": p, "q": q, "tokens": tokens, "u": torch.rand(N, generator=g, device="cuda"), "u_next": torch.rand(S, generator=g, device="cuda"), "V": V,
              "accepted": torch.empty(S, dtype=torch.int32, device="cuda"), "next": torch.empty(S, dtype=torch.int32, device="cuda"),
              "count": torch.empty(S, dtype=torch.int32, device="cuda")}
        if own:
            s["dims"] = s["G"].GdnDims.make(S, N, 1, 1, 1, 128, min(64, max(new)))
        return s

    t, d, page, hkv = TYPES[c["type"]], c["d"], c["page"], c["hkv"]
    need = [-(-(a + b) // page) for a, b in zip(ctx, new)]
    width, pages, layers = max(need), sum(need) + 3, c.get("layers", 1)
    perm = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    table, at = torch.zeros(S, width, dtype=torch.int32, device="cuda"), 0
    for k in range(S):
        table[k, :need[k]] = perm[at:at + need[k]]
        at += need[k]
    shape = (layers, pages, page, hkv, d)
    s |= {"table": table, "ctx_len": _i32(ctx), "ctx": ctx, "k_pool": normal(*shape, dtype=t), "v_pool": normal(*shape, dtype=t)}
    if c["op"] == "move":
        s |= {"accepted": _i32(acc), "new_len": torch.empty(S, dtype=torch.int32, device="cuda"), "layers": layers}
    else:
        s["q"] = normal(N, c["hq"] * d, dtype=t)
    if c["op"] == "append":
        half = c["rot"] // 2
        s |= {"k": normal(N, hkv * d, dtype=t), "v": normal(N, hkv * d, dtype=t), "q_out": torch.empty(N, c["hq"] * d, device="cuda", dtype=t),
              "q_norm": 1 + normal(d, std=0.1) if c["norm"] else None, "k_norm": 1 + normal(d, std=0.1) if c["norm"] else None,
              "inv_freq": torch.tensor([1e7 ** (-i / half) for i in range(half)], dtype=torch.float64, device="cuda"),
              "axis": _i32([i % c["axes"] for i in range(half)]),
              "pos": torch.randint(0, 200000, (N, c["axes"]), generator=g, device="cuda", dtype=torch.int32)}
    if c["op"] == "attend":
        s["o"] = torch.empty(N, c["hq"] * d, device="cuda", dtype=t)
    if own:
        G = s["G"]
        s["dims"] = G.AttnDims.make(S, N, max(new), c.get("hq", hkv), hkv, d, G.GDN_BF16 if c["type"] == "bf16" else G.GDN_FP16, pages, page, width)
        if c["op"] == "attend":
            s["work"] = torch.empty(G.gdn_attention_workspace_bytes(s["dims"]), dtype=torch.uint8, device="cuda")
    return s


# ---- one pass -----------------------------------------------------------------------------------------------------------------------


def run(s):
    return {"attend": _attend, "append": _append, "move": _move, "accept": _accept}[s["case"]["op"]](s)


def _places(s):
    """Each new token's sequence, its index in it, and its row in the pools seen as [pages * page]."""
    N, page = s["off"][-1], s["case"]["page"]
    n = torch.arange(N, device="cuda")
    seq = torch.searchsorted(s["node_off"][1:].long(), n, right=True)
    i = n - s["node_off"].long()[seq]
    at = s["ctx_len"].long()[seq] + i
    return seq, i, s["table"].long()[seq, at // page] * page + at % page


def _append(s):
    c = s["case"]
    if own:
        s["G"].gdn_rope_append(s["dims"], s["q"], c["hq"] * c["d"], s["k"], c["hkv"] * c["d"], s["v"], c["hkv"] * c["d"], s["q_norm"], s["k_norm"], 1e-6, s["pos"],
                               c["axes"], s["inv_freq"], s["axis"], c["rot"], 0, s["node_off"], s["ctx_len"], s["table"], s["q_out"], c["hq"] * c["d"],
                               s["k_pool"], s["v_pool"], s["status"])
        return s["q_out"], s["k_pool"], s["v_pool"]
    d, rot, N = c["d"], c["rot"], s["off"][-1]
    angle = s["pos"].double()[:, s["axis"].long()] * s["inv_freq"]
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]

    def turned(x, w):
        x = x.view(N, -1, d).float()
        if w is not None:
            x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * w
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        return torch.cat([a * cos - b * sin, b * cos + a * sin, x[..., rot:]], -1).to(s["q"].dtype)

    row = _places(s)[2]
    s["q_out"].copy_(turned(s["q"], s["q_norm"]).view(N, -1))
    s["k_pool"].view(-1, c["hkv"], d)[row] = turned(s["k"], s["k_norm"])
    s["v_pool"].view(-1, c["hkv"], d)[row] = s["v"].view(N, c["hkv"], d)
    return s["q_out"], s["k_pool"], s["v_pool"]


def _attend(s):
    c = s["case"]
    d, hq, hkv, page = c["d"], c["hq"], c["hkv"], c["page"]
    scale = d ** -0.5
    if own:
        s["G"].gdn_paged_attention(s["dims"], s["q"], hq * d, s["k_pool"], s["v_pool"], s["table"], s["ctx_len"], s["node_off"],
                                   s["parents"] if c["tree"] else None, scale, s["o"], s["work"], s["work"].numel(), s["status"])
        return s["o"]
    S, T, G = c["seqs"], max(s["new"]), hq // hkv
    L = max(a + b for a, b in zip(s["ctx"], s["new"]))
    ctx, new, off = s["ctx_len"].long(), (s["node_off"][1:] - s["node_off"][:-1]).long(), s["node_off"].long()
    j, i = torch.arange(L, device="cuda"), torch.arange(T, device="cuda")
    rows = (s["table"].long()[:, j // page] * page + j % page)  # [S][L]
    token = (off[:-1, None] + i).clamp(max=s["off"][-1] - 1)  # [S][T], the padding reads a row that is not used
    q = s["q"].view(-1, hkv, G, d)[token].permute(0, 2, 3, 1, 4).reshape(S, hkv, G * T, d).float()
    rel = j[None] - ctx[:, None]  # [S][L]: place among the new tokens
    if c["tree"]:
        parent = torch.where(i < new[:, None], s["parents"].long()[token], -1)
        one = (parent[..., None] == i).float()  # [S][T][T]: t's parent
        line = torch.linalg.matrix_power(one + torch.eye(T, device="cuda"), T) > 0  # ancestors and the token itself
        seen = torch.gather(line, 2, rel.clamp(0, T - 1)[:, None].expand(S, T, L)) & (rel < T)[:, None]
    else:
        seen = rel[:, None] <= i[None, :, None]
    seen = (seen | (rel < 0)[:, None]) & (j < (ctx + new)[:, None])[:, None]  # [S][T][L]
    k = s["k_pool"].view(-1, hkv, d)[rows].permute(0, 2, 1, 3).float()
    x = torch.matmul(q, k.transpose(2, 3)).mul_(scale).view(S, hkv, G, T, L)
    del k
    x.masked_fill_(~seen[:, None, None], -math.inf)
    x.sub_(x.amax(-1, keepdim=True).clamp_(min=-1e30)).exp_()
    total = x.sum(-1, keepdim=True)
    v = s["v_pool"].view(-1, hkv, d)[rows].permute(0, 2, 1, 3).float()
    o = torch.matmul(x.view(S, hkv, G * T, L), v).view(S, hkv, G, T, d) / total
    real = (i < new[:, None]).view(-1)
    s["o"].copy_(o.permute(0, 3, 1, 2, 4).reshape(S * T, hq * d)[real.nonzero().squeeze(1)] if c["ragged"] else o.permute(0, 3, 1, 2, 4).reshape(S * T, hq * d))
    return s["o"]


def _move(s):
    c = s["case"]
    if own:
        s["G"].gdn_kv_commit(s["dims"], s["layers"], s["k_pool"].stride(0), s["accepted"], s["parents"], s["node_off"], s["ctx_len"], s["table"], s["k_pool"],
                             s["v_pool"], s["new_len"], s["status"])
        return s["k_pool"], s["v_pool"], s["new_len"]
    seq, i, row = _places(s)
    N, T = s["off"][-1], max(s["new"])
    t, off = torch.arange(T, device="cuda"), s["node_off"].long()
    parent = s["parents"].long()
    one = (parent[:, None] == t).float()  # [N][T]
    per = one.view(c["seqs"], T, T) + torch.eye(T, device="cuda")
    line = torch.linalg.matrix_power(per, T) > 0  # ancestors and the node itself
    path = line[torch.arange(c["seqs"], device="cuda"), s["accepted"].long()]  # [S][T] the nodes of the accepted path
    place = path.long().cumsum(1) - 1
    on = path.view(-1).nonzero().squeeze(1)
    source = row[on]
    target_at = s["ctx_len"].long()[seq[on]] + place.view(-1)[on]
    target = s["table"].long()[seq[on], target_at // c["page"]] * c["page"] + target_at % c["page"]
    k, v = s["k_pool"].view(s["layers"], -1, c["hkv"] * c["d"]), s["v_pool"].view(s["layers"], -1, c["hkv"] * c["d"])
    k[:, target] = k[:, source]
    v[:, target] = v[:, source]
    s["new_len"].copy_(s["ctx_len"] + path.sum(1))
    return s["k_pool"], s["v_pool"], s["new_len"]


def _accept(s):
    c = s["case"]
    V = s["V"]
    if own:
        s["G"].gdn_tree_accept(s["dims"], V, s["p"], s["p"].stride(0), s["q"], s["q"].stride(0) if s["q"] is not None else 0, int(c["draft"] == "with"),
                               s["tokens"], s["parents"], s["node_off"], s["u"], s["u_next"], s["accepted"], s["next"], s["count"], s["status"])
        return s["accepted"], s["next"], s["count"]
    # A node's target distribution after its first k children were turned down is (p - c q)+ / W, with c and W from the ones before.
    # All in 64 bits: comparisons and the place in a cumulative sum stand next to borders.
    S, T = c["seqs"], max(s["new"])
    off, new = s["node_off"].long()[:-1], (s["node_off"][1:] - s["node_off"][:-1]).long()
    k = torch.arange(S, device="cuda")
    cur = torch.zeros(S, dtype=torch.long, device="cuda")
    depth = torch.ones(S, dtype=torch.long, device="cuda")
    cq, W, Z = (torch.full((S,), x, dtype=torch.float64, device="cuda") for x in (0.0, 1.0, 1.0))
    gone = torch.zeros(S, V, dtype=torch.bool, device="cuda")

    def rest(cur, cq, gone):
        p = s["p"][off + cur, :V].double()
        if s["q"] is not None:
            p = (p - cq[:, None] * s["q"][off + cur, :V].double()).clamp_(min=0)
        return p.masked_fill_(gone, 0.0)

    for t in range(1, T):  # children come after their parents and in the order in which they are tried
        row = (off + t).clamp(max=s["off"][-1] - 1)
        tries = (t < new) & (s["parents"].long()[row] == cur) & (Z > 0)  # a draft with nothing left has proposed nothing more
        x = s["tokens"].long()[row]
        u = s["u"][row].double()
        left = rest(cur, cq, gone)
        px = left[k, x]
        qx = s["q"][off + cur, x].double().masked_fill(gone[k, x], 0.0) if s["q"] is not None else torch.ones_like(px)
        yes = tries & (u * qx * W < px * Z)
        no = tries & ~yes
        if s["q"] is None or c["draft"] != "with":
            gone[k, x] |= no
        if s["q"] is not None:
            cq = torch.where(no, cq + W / Z, cq)
            if c["draft"] != "with":
                Z = torch.where(no, (Z - qx).clamp(min=0), Z)
            W = torch.where(no, rest(cur, cq, gone).sum(1), W)
        else:
            W = torch.where(no, (W - px).clamp(min=0), W)
        cur, depth = torch.where(yes, t, cur), depth + yes.long()
        cq, W, Z = (torch.where(yes, start, v) for start, v in ((0.0, cq), (1.0, W), (1.0, Z)))
        gone &= ~yes[:, None]
    left = rest(cur, cq, gone)
    none = (left.sum(1) <= 0)[:, None]  # nothing is left: the target's own row
    left = torch.where(none, s["p"][off + cur, :V].double(), left)
    sums = left.cumsum(1)
    s["accepted"].copy_(cur)
    s["next"].copy_(torch.searchsorted(sums, (s["u_next"].double() * sums[:, -1])[:, None], right=True).squeeze(1).clamp_(max=V - 1))
    s["count"].copy_(depth)
    return s["accepted"], s["next"], s["count"]


# ---- the definitions in 64 bits ---------------------------------------------------------------------------------------------------


def exact(c, seed):
    global own
    if c["op"] == "accept":
        return None  # whole numbers
    was, own = own, False
    try:
        s = prepare(c, seed)
    finally:
        own = was
    new, ctx, par, acc = _structure(c)
    page, d, hkv = c["page"], c["d"], c["hkv"]

    def rows(k, lo, hi):
        at = torch.arange(lo, hi, device="cuda")
        return s["table"][k].long()[torch.div(at, page, rounding_mode="floor")] * page + torch.remainder(at, page)

    if c["op"] == "move":
        pools = []
        for pool in (s["k_pool"], s["v_pool"]):
            flat = pool.double().reshape(c["layers"], -1, hkv * d)
            for k in range(c["seqs"]):
                way = _path(par[k], acc[k])
                place = rows(k, ctx[k], ctx[k] + new[k])
                flat[:, place[:len(way)]] = flat[:, place[torch.tensor(way, device="cuda")]].clone()
            pools.append(flat.view(pool.shape))
        return pools[0], pools[1], None
    if c["op"] == "append":
        half, rot = c["rot"] // 2, c["rot"]
        q = s["q"].double().view(-1, c["hq"], d)
        k = s["k"].double().view(-1, hkv, d)
        if c["norm"]:
            q = q / (q.pow(2).sum(-1, keepdim=True) / d + 1e-6).sqrt() * s["q_norm"].double()
            k = k / (k.pow(2).sum(-1, keepdim=True) / d + 1e-6).sqrt() * s["k_norm"].double()
        out = []
        for x in (q, k):
            z = torch.complex(x[..., :half].contiguous(), x[..., half:rot].contiguous())
            phi = torch.stack([s["pos"][:, i % c["axes"]].double() * s["inv_freq"][i] for i in range(half)], 1)
            z = z * torch.polar(torch.ones_like(phi), phi)[:, None]
            out.append(torch.cat([z.real, z.imag, x[..., rot:]], -1))
        kp, vp = s["k_pool"].double().reshape(-1, hkv, d), s["v_pool"].double().reshape(-1, hkv, d)
        for n in range(c["seqs"]):
            place = rows(n, ctx[n], ctx[n] + new[n])
            kp[place] = out[1][s["off"][n]:s["off"][n + 1]]
            vp[place] = s["v"].double().view(-1, hkv, d)[s["off"][n]:s["off"][n + 1]]
        return out[0].reshape(s["q"].shape), kp.view(s["k_pool"].shape), vp.view(s["v_pool"].shape)
    group = c["hq"] // hkv
    o = torch.empty(sum(new), c["hq"], d, dtype=torch.float64, device="cuda")
    for n in range(c["seqs"]):
        a, b = s["off"][n], s["off"][n + 1]
        place = rows(n, 0, ctx[n] + new[n])
        allowed = torch.ones(new[n], ctx[n] + new[n], dtype=torch.bool, device="cuda")
        if c["tree"]:
            line = torch.zeros(new[n], new[n], dtype=torch.bool)
            for i in range(new[n]):
                line[i, _path(par[n], i)] = True
            allowed[:, ctx[n]:] = line.cuda()
        else:
            allowed[:, ctx[n]:] = torch.ones(new[n], new[n], dtype=torch.bool, device="cuda").tril()
        for h in range(hkv):
            key, value = (pool.view(-1, hkv, d)[place, h].double() for pool in (s["k_pool"], s["v_pool"]))
            for e in range(h * group, (h + 1) * group):
                x = s["q"][a:b].view(-1, c["hq"], d)[:, e].double() @ key.T / math.sqrt(d)
                o[a:b, e] = torch.softmax(x.masked_fill(~allowed, -math.inf), 1) @ value
    return o.view(-1, c["hq"] * d)
