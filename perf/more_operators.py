"""Measured cases of a speculative round over a cache held in 4 bits, and of the sampling that goes with it.

Operators around one paged key/value cache of 4-bit values with a scale per 16 of them, and one token history:

  append   the new tokens' keys and values quantised into the cache, and read back as what the cache then holds
  attend   attention of a chunk of new tokens (a prompt chunk, a token tree, one token) over the 4-bit cache
  move     the accepted path's rows to their final places, for every layer at once, and read back
  probs    logits of a token tree to probabilities: penalties for repeated tokens (along each node's own path),
           biases, grammar masks, temperature, softmax
  tokens   the accepted path's tokens (or a prompt's) into the history that the penalties read

The cache.  A block (page, head) is `page` rows of d / 2 bytes of e2m1 codes (element 2 i in the low half of byte i),
then `page` rows of d / 16 scales in e4m3.  16 values x have the scale s = e4m3(max |x| / 6 unit) and the codes
e2m1(x / (s unit)), both to nearest even; they stand for code * s * unit.

`own = False` computes them in elementary torch operations; `own = True` calls the library's entry points.
Lengths, trees and accepted nodes follow from the case; values, tokens and the page order from the seed.
"""
import math
import random

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ---- cases ------------------------------------------------------------------------------------------------------------------


def listed():
    return [
        # one user, one token: the smallest call, where latency counts
        {"name": "attend4_one_token", "op": "attend", "type": "bf16", "seqs": 1, "new": 1, "ragged": False, "tree": False, "ctx": 777, "hq": 16, "hkv": 2,
         "d": 256, "page": 16, "unit": 1.0},
        # a full batch of plain decode steps over contexts of very different lengths: what a 4-bit cache is for
        {"name": "attend4_decode_batch", "op": "attend", "type": "bf16", "seqs": 64, "new": 1, "ragged": False, "tree": False, "ctx": 16384, "hq": 16,
         "hkv": 2, "d": 256, "page": 64, "unit": 1.0},
        # the headline round: 64 sequences of 16-node trees, here in the full-attention layer
        {"name": "attend4_trees", "op": "attend", "type": "bf16", "seqs": 64, "new": 16, "ragged": False, "tree": True, "ctx": 8192, "hq": 16, "hkv": 2,
         "d": 256, "page": 32, "unit": 1.0},
        # chunks of several prompts in one call, odd lengths, the other type and head width
        {"name": "attend4_mixed_chunks", "op": "attend", "type": "fp16", "seqs": 9, "new": 701, "ragged": True, "tree": False, "ctx": 3001, "hq": 32, "hkv": 8,
         "d": 128, "page": 16, "unit": 0.25},
        # a round's few new tokens
        {"name": "append4_trees", "op": "append", "type": "bf16", "seqs": 4, "new": 16, "ragged": False, "tree": True, "ctx": 1000, "hkv": 2, "d": 256,
         "page": 32, "unit": 1.0},
        # prompts of odd lengths
        {"name": "append4_prompt", "op": "append", "type": "bf16", "seqs": 3, "new": 4001, "ragged": True, "tree": False, "ctx": 50, "hkv": 2, "d": 256,
         "page": 64, "unit": 1.0},
        # one layer, few sequences; and all the attention layers of a stack for the headline batch
        {"name": "move4_one_layer", "op": "move", "type": "bf16", "seqs": 4, "new": 16, "ragged": False, "tree": True, "ctx": 500, "hkv": 2, "d": 256,
         "page": 16, "layers": 1, "unit": 1.0},
        {"name": "move4_stack", "op": "move", "type": "bf16", "seqs": 64, "new": 16, "ragged": False, "tree": True, "ctx": 500, "hkv": 2, "d": 256, "page": 32,
         "layers": 12, "unit": 1.0},
        # one user's tree; the headline batch with penalties, biases and a grammar for half of the sequences
        {"name": "probs_one_tree", "op": "probs", "type": "bf16", "seqs": 1, "new": 16, "ragged": False, "tree": True, "vocab": 131072, "bias": 5, "grammar": True},
        {"name": "probs_trees", "op": "probs", "type": "bf16", "seqs": 64, "new": 16, "ragged": False, "tree": True, "vocab": 131072, "bias": 40,
         "grammar": True},
        # the headline batch's accepted paths; prompts that begin
        {"name": "tokens_round", "op": "tokens", "seqs": 64, "new": 16, "ragged": False, "tree": True, "vocab": 131072, "prompt": False},
        {"name": "tokens_prompts", "op": "tokens", "seqs": 8, "new": 4001, "ragged": True, "tree": False, "vocab": 131072, "prompt": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attend", "attend", "attend", "append", "move", "probs", "probs", "tokens"])
    if op == "probs":
        return {"op": op, "type": rng.choice(["bf16", "fp16", "fp32"]), "seqs": _log(rng, 1, 48), "new": rng.randint(1, 16), "ragged": rng.random() < 0.5,
                "tree": rng.random() < 0.7, "vocab": _log(rng, 1000, 131072), "bias": rng.choice([0, rng.randint(1, 100)]), "grammar": rng.random() < 0.5}
    if op == "tokens":
        prompt = rng.random() < 0.4
        return {"op": op, "seqs": _log(rng, 1, 64), "new": _log(rng, 2, 2000) if prompt else rng.randint(1, 32), "ragged": rng.random() < 0.5,
                "tree": not prompt and rng.random() < 0.7, "vocab": _log(rng, 1000, 131072), "prompt": prompt}
    d, hkv, group = rng.choice([(256, 2, 8), (256, 4, 4), (256, 2, 6), (128, 8, 4), (128, 4, 5), (64, 8, 1)])
    c = {"op": op, "type": rng.choice(["bf16", "fp16"]), "hkv": hkv, "d": d, "page": rng.choice([16, 32, 64, 128]), "unit": 2.0 ** rng.randint(-4, 2)}
    if op == "move":
        return {**c, "seqs": _log(rng, 1, 64), "new": rng.randint(2, 32), "ragged": rng.random() < 0.5, "tree": rng.random() < 0.7, "ctx": _log(rng, 1, 500),
                "layers": rng.randint(1, 12)}
    if op == "attend":
        c["hq"] = hkv * group
    kind = rng.choice(["decode", "tree", "chunk"])
    if kind == "decode":
        return {**c, "seqs": _log(rng, 1, 64), "new": 1, "ragged": False, "tree": False, "ctx": _log(rng, 1, 12000)}
    if kind == "tree":
        return {**c, "seqs": _log(rng, 1, 48), "new": rng.randint(2, 40), "ragged": rng.random() < 0.5, "tree": True, "ctx": _log(rng, 1, 5000)}
    return {**c, "seqs": rng.randint(1, 5), "new": _log(rng, 17, 1200), "ragged": True, "tree": False, "ctx": _log(rng, 1, 4000)}


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
    new = [max(1, n - (i * n) // (2 * S)) if c["ragged"] else n for i in range(S)]
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
    if c["op"] == "tokens":
        n = N if c["prompt"] else sum(len(_path(p, a)) for p, a in zip(par, acc))
        return {"bytes": 4 * n + 2 * 2 * n, "flops": 0}
    if c["op"] == "probs":
        V = c["vocab"]
        size = 4 if c["type"] == "fp32" else 2
        rows = sum(k for s, k in enumerate(new) if s % 2 == 0) if c["grammar"] else 0
        return {"bytes": N * V * (size + 4) + c["seqs"] * V * 2 + rows * V // 8, "flops": 6 * N * V}
    row = c["d"] * 9 // 16  # a token's keys (or values) of one head: codes and scales
    if c["op"] == "move":  # the moved rows read and written, and the sequences' new rows read back in 16 bits
        moved = sum(1 for p, a in zip(par, acc) for j, x in enumerate(_path(p, a)) if x != j)
        return {"bytes": (moved * 2 * row + N * (row + 2 * c["d"])) * 2 * c["hkv"] * c["layers"], "flops": 0}
    if c["op"] == "append":  # 16-bit rows in, 4-bit rows out and in, 16-bit rows out
        return {"bytes": N * 2 * c["hkv"] * (4 * c["d"] + 2 * row), "flops": 0}
    seen = [sum(ctx[s] + (len(_path(par[s], i)) if c["tree"] else i + 1) for i in range(new[s])) for s in range(c["seqs"])]
    return {"bytes": sum((a + b) for a, b in zip(ctx, new)) * 2 * c["hkv"] * row + 2 * 2 * N * c["hq"] * c["d"], "flops": 4 * c["d"] * c["hq"] * sum(seen)}


# ---- the cache's values in elementary operations ------------------------------------------------------------------------------


def _quantise(x, unit):
    """[..., d] values as codes [..., d / 2] and scales [..., d / 16], both uint8."""
    x = x.float().unflatten(-1, (-1, 16))
    # in 64 bits: 16-bit values often stand on the border of two scales
    s = (x.abs().amax(-1).double() / (6 * unit)).clamp_(max=448).float().to(torch.float8_e4m3fn)
    sf = s.float()[..., None] * unit
    t = torch.where(sf > 0, x.abs() / sf, 0)
    code = (t > 0.25).to(torch.uint8)
    for border, tie in ((0.75, True), (1.25, False), (1.75, True), (2.5, False), (3.5, True), (5.0, False)):
        code += (t >= border) if tie else (t > border)
    code = (code + 8 * (x < 0).to(torch.uint8)).flatten(-2)
    return code[..., 0::2] + 16 * code[..., 1::2], s.view(torch.uint8)


def _values(codes, scales, unit):
    """What codes [..., d / 2] and scales [..., d / 16] stand for, in 32 bits."""
    lut = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, 0, -0.5, -1, -1.5, -2, -3, -4, -6], device=codes.device)
    c = torch.stack([codes & 15, codes >> 4], -1).flatten(-2)
    s = scales.view(torch.float8_e4m3fn).float() * unit
    return (lut[c.int()].unflatten(-1, (-1, 16)) * s[..., None]).flatten(-2)


def _parts(pool, c):
    """Views of a pool [..., pages, heads, bytes]: codes [..., pages, heads, page, d / 2] and scales [..., pages, heads, page, d / 16]."""
    n = c["page"] * c["d"] // 2
    return pool[..., :n].unflatten(-1, (c["page"], -1)), pool[..., n:].unflatten(-1, (c["page"], -1))


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
         "parents": _i32([x for p in par for x in p]) if par else None, "accepted": _i32(acc) if acc else None}
    if own:
        import gated_deltanet_speculative_gdn_gb300 as G
        s["G"] = G
    if c["op"] in ("probs", "tokens"):
        V, P = c["vocab"], (c["vocab"] + 7) // 8 * 8
        # tokens as text has them: few of them often
        def text(*shape):
            return (V * torch.rand(shape, generator=g, device="cuda", dtype=torch.float64) ** 4).to(torch.int32).clamp_(max=V - 1)

        slots = S + 3
        history = torch.zeros(slots, P, dtype=torch.int16, device="cuda")  # bits 0 .. 14: how often produced, bit 15: in the prompt
        history.scatter_add_(1, text(slots, 300).long(), torch.ones(slots, 300, dtype=torch.int16, device="cuda"))
        history.scatter_(1, text(slots, 1000).long(), -32768)
        s |= {"history": history, "slot_map": torch.randperm(slots, generator=g, device="cuda")[:S].to(torch.int32), "tokens": text(N)}
        if own:
            s["dims"] = G.GdnDims.make(S, N, slots, 1, 1, 128, min(64, max(new)))
        if c["op"] == "tokens":
            return s
        size = (V + 31) // 32
        words = torch.randint(-2 ** 31, 2 ** 31, (N, size), generator=g, device="cuda", dtype=torch.int64).to(torch.int32)
        seq = torch.repeat_interleave(torch.arange(S, device="cuda"), torch.tensor(new, device="cuda"))
        r = torch.rand(4, S, generator=g, device="cuda")
        s |= {"logits": torch.zeros(N, P, dtype=TYPES[c["type"]], device="cuda"), "p": torch.zeros(N, P, device="cuda"),
              # a grammar for every other sequence: half of the tokens are allowed
              "mask": words if c["grammar"] else None, "mask_row": torch.where(seq % 2 == 0, torch.arange(N, device="cuda"), -1).to(torch.int32),
              "repetition": 1 + 0.3 * r[0], "frequency": 0.5 * r[1], "presence": 0.5 * r[2],
              # every eighth sequence takes the most probable token
              "temperature": torch.where(torch.arange(S, device="cuda") % 8 == 5, torch.zeros(S, device="cuda"), 0.5 + 0.7 * r[3])}
        s["logits"][:, :V] = normal(N, V, std=3.0)
        k = min(c["bias"], V // 2)
        if k:  # a list of tokens for each sequence, in ascending order
            s["bias_off"] = _i32([k * i for i in range(S + 1)])
            s["bias_token"] = torch.rand(S, V, generator=g, device="cuda").topk(k, dim=1).indices.sort(dim=1).values.to(torch.int32).view(-1)
            s["bias_value"] = normal(S * k, std=4.0)
        return s

    t, d, page, hkv = TYPES[c["type"]], c["d"], c["page"], c["hkv"]
    need = [-(-(a + b) // page) for a, b in zip(ctx, new)]
    width, pages, layers = max(need), sum(need) + 3, c.get("layers", 1)
    perm = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    table, at = torch.zeros(S, width, dtype=torch.int32, device="cuda"), 0
    for k in range(S):
        table[k, :need[k]] = perm[at:at + need[k]]
        at += need[k]
    s |= {"table": table, "ctx_len": _i32(ctx), "ctx": ctx}
    for name in ("k_pool", "v_pool"):
        s[name] = torch.empty(layers, pages, hkv, page * d * 9 // 16, dtype=torch.uint8, device="cuda")
        codes, scales = _parts(s[name], c)
        for x in range(layers):
            for y in range(0, pages, 4096):
                n = min(4096, pages - y)
                codes[x, y:y + n], scales[x, y:y + n] = _quantise(normal(n, hkv, page, d, dtype=t), c["unit"])
    if c["op"] == "attend":
        s |= {"q": normal(N, c["hq"] * d, dtype=t), "o": torch.empty(N, c["hq"] * d, device="cuda", dtype=t)}
    else:
        s |= {"k": normal(N, hkv * d, dtype=t), "v": normal(N, hkv * d, dtype=t), "layers": layers,
              "k_out": torch.empty(layers, N, hkv * d, device="cuda", dtype=t), "v_out": torch.empty(layers, N, hkv * d, device="cuda", dtype=t),
              "new_len": torch.empty(S, dtype=torch.int32, device="cuda")}
    if own:
        s["dims"] = G.AttnDims.make_kvq(S, N, max(new), c.get("hq", hkv), hkv, d, G.GDN_BF16 if c["type"] == "bf16" else G.GDN_FP16, pages, page, width)
        if c["op"] == "attend":
            s["work"] = torch.empty(G.gdn_attention_kvq_workspace_bytes(s["dims"]), dtype=torch.uint8, device="cuda")
    return s


# ---- one pass -----------------------------------------------------------------------------------------------------------------------


def run(s):
    return {"attend": _attend, "append": _append, "move": _move, "probs": _probs, "tokens": _tokens}[s["case"]["op"]](s)


def _places(s):
    """Each new token's sequence, its index in it, and its page and place in the page."""
    N, page = s["off"][-1], s["case"]["page"]
    n = torch.arange(N, device="cuda")
    seq = torch.searchsorted(s["node_off"][1:].long(), n, right=True)
    i = n - s["node_off"].long()[seq]
    at = s["ctx_len"].long()[seq] + i
    return seq, i, s["table"].long()[seq, at // page], at % page


def _read(s):
    """The new tokens' rows as the cache holds them."""
    c = s["case"]
    if own:
        s["G"].gdn_kvq_read(s["dims"], s["layers"], s["k_pool"].stride(0), s["k_pool"], s["v_pool"], c["unit"], c["unit"], s["node_off"], s["ctx_len"],
                            s["table"], s["k_out"], s["v_out"], c["hkv"] * c["d"], s["status"])
        return s["k_out"], s["v_out"]
    page, at = _places(s)[2:]
    for pool, out in ((s["k_pool"], s["k_out"]), (s["v_pool"], s["v_out"])):
        codes, scales = _parts(pool, c)
        x = _values(codes[:, page, :, at], scales[:, page, :, at], c["unit"])  # [token][layer][head][d]
        out.copy_(x.transpose(0, 1).flatten(2))
    return s["k_out"], s["v_out"]


def _append(s):
    c = s["case"]
    if own:
        s["G"].gdn_kvq_append(s["dims"], s["k"], c["hkv"] * c["d"], s["v"], c["hkv"] * c["d"], c["unit"], c["unit"], s["node_off"], s["ctx_len"], s["table"],
                              s["k_pool"], s["v_pool"], s["status"])
        return _read(s)
    page, at = _places(s)[2:]
    for pool, x in ((s["k_pool"], s["k"]), (s["v_pool"], s["v"])):
        codes, scales = _parts(pool, c)
        codes[0, page, :, at], scales[0, page, :, at] = _quantise(x.view(-1, c["hkv"], c["d"]), c["unit"])
    return _read(s)


def _line(s):
    """[S][T][T]: which nodes of a sequence are a node's ancestors, or itself."""
    T = max(s["new"])
    i = torch.arange(T, device="cuda")
    off, new = s["node_off"].long()[:-1], (s["node_off"][1:] - s["node_off"][:-1]).long()
    token = (off[:, None] + i).clamp(max=s["off"][-1] - 1)  # the padding reads a row that is not used
    parent = torch.where(i < new[:, None], s["parents"].long()[token], -1)
    one = (parent[..., None] == i).float()
    return torch.linalg.matrix_power(one + torch.eye(T, device="cuda"), T) > 0


def _attend(s):
    c = s["case"]
    d, hq, hkv, page = c["d"], c["hq"], c["hkv"], c["page"]
    scale = d ** -0.5
    if own:
        s["G"].gdn_paged_attention_kvq(s["dims"], s["q"], hq * d, s["k_pool"], s["v_pool"], c["unit"], c["unit"], s["table"], s["ctx_len"], s["node_off"],
                                       s["parents"] if c["tree"] else None, scale, s["o"], s["work"], s["work"].numel(), s["status"])
        return s["o"]
    S, T, G = c["seqs"], max(s["new"]), hq // hkv
    L = max(a + b for a, b in zip(s["ctx"], s["new"]))
    ctx, new, off = s["ctx_len"].long(), (s["node_off"][1:] - s["node_off"][:-1]).long(), s["node_off"].long()
    j, i = torch.arange(L, device="cuda"), torch.arange(T, device="cuda")
    token = (off[:-1, None] + i).clamp(max=s["off"][-1] - 1)  # [S][T], the padding reads a row that is not used
    q = s["q"].view(-1, hkv, G, d)[token].permute(0, 2, 3, 1, 4).reshape(S, hkv, G * T, d).float()
    rel = j[None] - ctx[:, None]  # [S][L]: place among the new tokens
    if c["tree"]:
        seen = torch.gather(_line(s), 2, rel.clamp(0, T - 1)[:, None].expand(S, T, L)) & (rel < T)[:, None]
    else:
        seen = rel[:, None] <= i[None, :, None]
    seen = (seen | (rel < 0)[:, None]) & (j < (ctx + new)[:, None])[:, None]  # [S][T][L]

    def cached(pool):  # [S][heads][L][d]
        codes, scales = (x[0].transpose(1, 2) for x in _parts(pool, c))
        at = s["table"].long()[:, j // page]
        return _values(codes[at, j % page], scales[at, j % page], c["unit"]).transpose(1, 2)

    x = torch.matmul(q, cached(s["k_pool"]).transpose(2, 3)).mul_(scale).view(S, hkv, G, T, L)
    x.masked_fill_(~seen[:, None, None], -math.inf)
    x.sub_(x.amax(-1, keepdim=True).clamp_(min=-1e30)).exp_()
    total = x.sum(-1, keepdim=True)
    o = torch.matmul(x.view(S, hkv, G * T, L), cached(s["v_pool"])).view(S, hkv, G, T, d) / total
    real = (i < new[:, None]).view(-1)
    o = o.permute(0, 3, 1, 2, 4).reshape(S * T, hq * d)
    s["o"].copy_(o[real.nonzero().squeeze(1)] if c["ragged"] else o)
    return s["o"]


def _move(s):
    c = s["case"]
    if own:
        s["G"].gdn_kvq_commit(s["dims"], s["layers"], s["k_pool"].stride(0), s["accepted"], s["parents"], s["node_off"], s["ctx_len"], s["table"], s["k_pool"],
                              s["v_pool"], s["new_len"], s["status"])
        return _read(s) + (s["new_len"],)
    seq, i, page, place = _places(s)
    path = _line(s)[torch.arange(c["seqs"], device="cuda"), s["accepted"].long()]  # [S][T] the nodes of the accepted path
    nth = path.long().cumsum(1) - 1
    who, node = path.nonzero(as_tuple=True)
    source = s["node_off"].long()[who] + node
    target = s["node_off"].long()[who] + nth[who, node]
    for pool in (s["k_pool"], s["v_pool"]):
        for x in _parts(pool, c):
            x[:, page[target], :, place[target]] = x[:, page[source], :, place[source]]
    s["new_len"].copy_(s["ctx_len"] + path.sum(1))
    return _read(s) + (s["new_len"],)


def _probs(s):
    c = s["case"]
    V = c["vocab"]
    if own:
        s["G"].gdn_logits_probs(s["dims"], V, {"bf16": s["G"].GDN_BF16, "fp16": s["G"].GDN_FP16, "fp32": s["G"].GDN_FP32}[c["type"]], s["logits"],
                                s["logits"].stride(0), s["tokens"], s["parents"], s["node_off"], s["slot_map"], s["history"], s["history"].stride(0),
                                s["repetition"], s["frequency"], s["presence"], s["temperature"], s.get("bias_off"), s.get("bias_token"), s.get("bias_value"),
                                s["bias_token"].numel() if "bias_token" in s else 0, s["mask"], s["mask"].stride(0) if s["mask"] is not None else 0,
                                s["mask_row"] if s["mask"] is not None else None, s["mask"].shape[0] if s["mask"] is not None else 0, s["p"],
                                s["p"].stride(0), s["status"])
        return s["p"]
    N = s["off"][-1]
    seq, i = _places_of_nodes(s)
    x = s["logits"][:, :V].float()
    past = s["history"].int()[s["slot_map"].long()][:, :V][seq]
    count, seen = past & 32767, past != 0
    who, node, up = _line(s).nonzero(as_tuple=True)  # (sequence, node, an ancestor or itself)
    real = (node < torch.tensor(s["new"], device="cuda")[who]).nonzero().squeeze(1)
    off = s["node_off"].long()[who[real]]
    count.index_put_((off + node[real], s["tokens"].long()[off + up[real]]), torch.ones_like(off, dtype=torch.int32), accumulate=True)
    seen |= count > 0
    r = s["repetition"][seq][:, None]
    x = torch.where(seen, torch.where(x > 0, x / r, x * r), x)
    x -= s["frequency"][seq][:, None] * count
    x -= s["presence"][seq][:, None] * (count > 0)
    if "bias_off" in s:
        each = s["bias_token"].long().view(c["seqs"], -1)[seq]
        x.scatter_add_(1, each, s["bias_value"].view(c["seqs"], -1)[seq])
    if s["mask"] is not None:
        bit = torch.arange(32, device="cuda", dtype=torch.int32)
        allowed = ((s["mask"][:, :, None] >> bit) & 1).bool().view(N, -1)[:, :V]
        x.masked_fill_(~allowed & (s["mask_row"] >= 0)[:, None], -math.inf)
    t = s["temperature"][seq][:, None]
    top, best = x.max(1, keepdim=True)
    e = torch.exp((x - top) / torch.where(t > 0, t, 1.0))
    e = torch.where(t > 0, e / e.sum(1, keepdim=True), (torch.arange(V, device="cuda") == best).float())
    s["p"][:, :V] = torch.where(top > -math.inf, e, 0.0)
    return s["p"]


def _places_of_nodes(s):
    n = torch.arange(s["off"][-1], device="cuda")
    seq = torch.searchsorted(s["node_off"][1:].long(), n, right=True)
    return seq, n - s["node_off"].long()[seq]


def _tokens(s):
    c = s["case"]
    if own:
        s["G"].gdn_token_commit(s["dims"], c["vocab"], s["tokens"], None if c["prompt"] else s["accepted"], None if c["prompt"] else s["parents"], s["node_off"],
                                s["slot_map"], int(c["prompt"]), s["history"], s["history"].stride(0), s["status"])
        return s["history"]
    seq, i = _places_of_nodes(s)
    row, token = s["slot_map"].long()[seq], s["tokens"].long()
    if c["prompt"]:
        s["history"][row, token] |= -32768
        return s["history"]
    on = _line(s)[torch.arange(c["seqs"], device="cuda"), s["accepted"].long()][seq, i].nonzero().squeeze(1)
    h = s["history"].int()
    count = (h & 32767).index_put_((row[on], token[on]), torch.ones_like(on, dtype=torch.int32), accumulate=True).clamp_(max=32767)
    s["history"].copy_(count | (h & 32768))
    return s["history"]


# ---- the definitions in 64 bits ---------------------------------------------------------------------------------------------------


def _meaning(codes, scales, unit):
    """Values in 64 bits from the formats' fields: e2m1 has a sign, two bits of exponent (bias 1) and one of fraction, e4m3 four (bias 7) and three."""
    both = torch.stack([codes.long() % 16, codes.long() // 16], -1).flatten(-2)
    e, f = (both // 2) % 4, (both % 2).double()
    x = torch.where(e > 0, (1 + f / 2) * torch.pow(2.0, e.double() - 1), f / 2) * (1 - 2 * (both // 8).double())
    b = scales.long()
    e, f = (b // 8) % 16, (b % 8).double()
    y = torch.where(e > 0, (1 + f / 8) * torch.pow(2.0, e.double() - 7), f / 8 * 2.0 ** -6) * (1 - 2 * (b // 128).double())
    return x * y.repeat_interleave(16, -1) * unit


def _to(grid, x):
    """The nearest of the ascending values `grid` to each x >= 0, a tie to the one with an even index."""
    mid = (grid[1:] + grid[:-1]) / 2
    i = torch.searchsorted(mid, x.contiguous())  # how many borders are below x
    return grid[torch.where((i < len(mid)) & (mid[i.clamp(max=len(mid) - 1)] == x) & (i % 2 == 1), i + 1, i)]


def _nearest(x, unit):
    """The values in 64 bits that the cache holds in the place of x: [..., d]."""
    e4m3 = torch.tensor([(1 + f / 8 if e else f / 8) * 2.0 ** (max(e, 1) - 7) for e in range(16) for f in range(8)][:-1], dtype=torch.float64, device=x.device)
    e2m1 = torch.tensor([(1 + f / 2 if e else f / 2) * 2.0 ** (max(e, 1) - 1) for e in range(4) for f in range(2)], dtype=torch.float64, device=x.device)
    x = x.double().unflatten(-1, (-1, 16)) / unit
    s = _to(6 * e4m3, x.abs().amax(-1, keepdim=True)) / 6  # (the borders times 6 are exact)
    t = torch.where(s > 0, _to(e2m1, x.abs() / s), 0)
    return (torch.copysign(t, x) * s * unit).flatten(-2)


def exact(c, seed):
    global own
    if c["op"] == "tokens":
        return None  # whole numbers
    was, own = own, False
    try:
        s = prepare(c, seed)
    finally:
        own = was
    new, ctx, par, acc = _structure(c)
    if c["op"] == "probs":
        V = c["vocab"]
        p = torch.zeros(s["p"].shape, dtype=torch.float64, device="cuda")
        words = s["mask"].cpu().numpy().view("uint32") if s["mask"] is not None else None
        tokens = s["tokens"].tolist()
        for k in range(c["seqs"]):
            past = s["history"][int(s["slot_map"][k]), :V].long() % 65536
            rep, freq, pres, temp = (float(s[x][k]) for x in ("repetition", "frequency", "presence", "temperature"))
            for n in range(new[k]):
                row = s["off"][k] + n
                made, known = past % 32768, past > 0
                for x in _path(par[k], n):
                    y = tokens[s["off"][k] + x]
                    made = made.clone() if x == 0 else made
                    made[y] += 1
                known = known | (made > 0)
                x = s["logits"][row, :V].double()
                x = torch.where(known & (x > 0), x / rep, torch.where(known, x * rep, x)) - freq * made - pres * (made > 0)
                if "bias_off" in s:
                    a, b = int(s["bias_off"][k]), int(s["bias_off"][k + 1])
                    x[s["bias_token"][a:b].long()] += s["bias_value"][a:b].double()
                if words is not None and k % 2 == 0:
                    import numpy
                    bits = numpy.unpackbits(words[row].view("uint8"), bitorder="little")[:V]
                    x = torch.where(torch.from_numpy(bits).cuda() > 0, x, -math.inf)
                if temp > 0:
                    p[row, :V] = torch.softmax(x / temp, 0)
                else:
                    p[row, int(x.argmax())] = 1.0
        return p
    d, hkv = c["d"], c["hkv"]

    def rows(k, lo, hi):
        at = torch.arange(lo, hi, device="cuda")
        return s["table"][k].long()[torch.div(at, c["page"], rounding_mode="floor")], torch.remainder(at, c["page"])

    if c["op"] == "append":
        return tuple(_nearest(s[x].view(-1, hkv, d), c["unit"]).view(1, -1, hkv * d) for x in ("k", "v"))
    if c["op"] == "move":
        out = []
        for pool in (s["k_pool"], s["v_pool"]):
            codes, scales = _parts(pool, c)
            each = []
            for k in range(c["seqs"]):
                page, at = rows(k, ctx[k], ctx[k] + new[k])
                x = _meaning(codes[:, page, :, at], scales[:, page, :, at], c["unit"])  # [token][layer][head][d]
                way = _path(par[k], acc[k])
                x[:len(way)] = x[torch.tensor(way, device="cuda")].clone()
                each.append(x.transpose(0, 1).flatten(2))
            out.append(torch.cat(each, 1))
        return out[0], out[1], None
    group = c["hq"] // hkv
    o = torch.empty(sum(new), c["hq"], d, dtype=torch.float64, device="cuda")
    for n in range(c["seqs"]):
        a, b = s["off"][n], s["off"][n + 1]
        page, at = rows(n, 0, ctx[n] + new[n])
        allowed = torch.ones(new[n], ctx[n] + new[n], dtype=torch.bool, device="cuda")
        if c["tree"]:
            line = torch.zeros(new[n], new[n], dtype=torch.bool)
            for i in range(new[n]):
                line[i, _path(par[n], i)] = True
            allowed[:, ctx[n]:] = line.cuda()
        else:
            allowed[:, ctx[n]:] = torch.ones(new[n], new[n], dtype=torch.bool, device="cuda").tril()
        for h in range(hkv):
            key, value = (_meaning(codes[0][page, h, at], scales[0][page, h, at], c["unit"]) for codes, scales in (_parts(s["k_pool"], c), _parts(s["v_pool"], c)))
            for e in range(h * group, (h + 1) * group):
                x = s["q"][a:b].view(-1, c["hq"], d)[:, e].double() @ key.T / math.sqrt(d)
                o[a:b, e] = torch.softmax(x.masked_fill(~allowed, -math.inf), 1) @ value
    return o.view(-1, c["hq"] * d)
