"""The cache operators of a decoder whose projections are 1-bit linear layers:
what runs between the QKV projection and the output projection, over one paged
key/value cache.

  rope    per-head RMS norm of queries and keys, position rotation, append of
          keys and values to the cache
  attn    attention of each sequence's drafted tokens (a tree, or a causal run;
          one token is plain decoding) over the cached tokens
  score   attention weight that each cached token received from the accepted
          tokens, added to its running sum
  evict   rejected drafts dropped and the cache cut to a budget by that sum

A cache is K, V [pages, page, kv heads, dim] (any strides) with a page table
[sequences, pages per sequence].  Sequence b holds ctx[b] committed tokens in
its slots 0 .. ctx[b]-1 and its drafted tokens in the slots after them.
"""
import math
import random

import numpy as np
import torch

own = False

KINDS = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
EPS = 1e-6


def listed():
    base = dict(seqs=1, nodes=1, ctx=0, heads=32, kv=8, dim=128, page=64, kind="bf16", order="token", ragged=False, tree=False)
    rope = dict(base, op="rope", src="f32", rot=128, interleaved=False, norm=True)
    attn = dict(base, op="attn", out="same", blank=False)
    score = dict(base, op="score", accepted=1)
    evict = dict(base, op="evict", accepted=1)
    return [
        # one new token of one conversation: latency
        dict(rope, name="rope_one_token", ctx=1000),
        # drafts of a small batch, part of the head rotated, interleaved pairs, odd counts, no norms
        dict(rope, name="rope_drafts_part", seqs=12, nodes=23, ctx=700, heads=20, kv=4, dim=96, page=16, kind="f16", order="head", ragged=True,
             tree=True, src="f16", rot=48, interleaved=True, norm=False),
        # prompts of a batch: 8190 tokens in 6 sequences
        dict(rope, name="rope_prompts", seqs=6, nodes=1365, ctx=0),
        # one new token of one conversation; fp32 out, as the INT8 quantizer of the next projection takes it
        dict(attn, name="attn_one_token", ctx=4000, out="f32"),
        # decoding of a full batch: the cache is read once
        dict(attn, name="attn_batch", seqs=64, ctx=8000, page=16, ragged=True),
        # drafted trees over long documents
        dict(attn, name="attn_trees_long", seqs=4, nodes=63, ctx=32000, order="head", tree=True),
        # a chunk of a prompt over what came before it
        dict(attn, name="attn_prompt_chunk", nodes=1024, ctx=8192, page=128),
        # small trees, a key head for each query head, short and empty contexts, a row that sees nothing
        dict(attn, name="attn_trees_short", seqs=9, nodes=13, ctx=517, heads=12, kv=12, dim=64, page=24, kind="f16", ragged=True, tree=True, blank=True),
        # the sums after one decoded token
        dict(score, name="score_one_token", ctx=4000),
        # the sums after verification of a batch of trees
        dict(score, name="score_trees", seqs=16, nodes=31, ctx=16000, page=16, order="head", ragged=True, tree=True, accepted=5),
        # every step of a batch: rejected drafts out, a few tokens over the budget
        dict(evict, name="evict_step", seqs=16, nodes=31, ctx=2048, page=16, order="head", ragged=True, tree=True, accepted=5, budget=2048, recent=256),
        # long prompts cut to a budget
        dict(evict, name="evict_prompts", seqs=4, nodes=1, ctx=32000, page=64, budget=4096, recent=512),
    ]


def spread(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    c = dict(op=rng.choice(("rope", "attn", "attn", "score", "evict")))
    c["seqs"] = spread(rng, 1, 64)
    c["nodes"] = rng.choice((1, spread(rng, 1, 64), spread(rng, 1, 64)))
    c["ctx"] = spread(rng, 60, 32000)
    c["kv"] = rng.choice((1, 2, 4, 5, 8, 16))
    c["heads"] = c["kv"] * rng.choice((1, 1, 2, 4, 5, 8))
    c["dim"] = rng.choice((64, 96, 128, 128, 256))
    c["page"] = rng.choice((1, 16, 24, 64, 128, 256))
    c["kind"] = rng.choice(("bf16", "bf16", "f16"))
    c["order"] = rng.choice(("token", "head"))
    c["ragged"] = rng.random() < 0.7
    c["tree"] = c["nodes"] > 1 and rng.random() < 0.8
    if c["op"] == "rope":
        if not c["tree"]:
            c["nodes"] = spread(rng, 1, 2000)
        c["src"] = rng.choice(("f32", "f32", c["kind"]))
        c["rot"] = rng.choice((c["dim"], c["dim"], c["dim"] // 2))
        c["interleaved"] = rng.random() < 0.4
        c["norm"] = rng.random() < 0.7
    elif c["op"] == "attn":
        if c["nodes"] > 1 and not c["tree"]:
            c["nodes"] = spread(rng, 2, 1000)
        c["out"] = rng.choice(("same", "same", "f32"))
        c["blank"] = c["tree"] and rng.random() < 0.3
    else:
        c["accepted"] = rng.randint(1, min(8, c["nodes"]))
    if c["op"] == "evict":
        c["budget"] = max(1, int(c["ctx"] * rng.uniform(0.05, 1.05)))
        c["recent"] = int(c["budget"] * rng.uniform(0, 0.6))

    def cost(x):
        w = work(x)
        rows, slots = x["seqs"] * x["nodes"] * x["heads"], x["ctx"] + x["nodes"]
        return max(w["bytes"] / 1.2e9, w["flops"] / 1.2e11, x["seqs"] * x["kv"] * x["dim"] * slots / 5e8, rows * slots / 2.5e8 if x["op"] != "rope" else 0)

    while cost(c) > 1:  # no dearer than the listed ones: fewer sequences first, then shorter ones
        if c["seqs"] > 1:
            c["seqs"] = c["seqs"] * 2 // 3
        elif c["ctx"] > 100:
            c["ctx"] = c["ctx"] * 2 // 3
        else:
            c["nodes"] = max(1, c["nodes"] * 2 // 3)
            c["tree"] = c["tree"] and c["nodes"] > 1
    if c["op"] == "evict":
        c["budget"] = min(c["budget"], c["ctx"] + c["accepted"])
        c["recent"] = min(c["recent"], c["budget"])
    return c


def lengths(case):
    """Committed and drafted tokens of each sequence."""
    n, ctx, nodes = case["seqs"], case["ctx"], case["nodes"]
    if not case["ragged"]:
        return [ctx] * n, [nodes] * n
    held = [ctx - ctx * (5 * b % 8) // 16 for b in range(n)]
    new = [max(1, nodes - b % 3) for b in range(n)]
    if n >= 4:
        held[1] = 0  # a conversation that begins
        new[2] = 0   # one that waits
    return held, new


def work(case):
    held, new = lengths(case)
    heads, kv, dim = case["heads"], case["kv"], case["dim"]
    rows = sum(new)
    if case["op"] == "rope":
        src = 4 if case["src"] == "f32" else 2
        values = rows * (heads + 2 * kv) * dim
        return {"bytes": values * (src + 2) + rows * (4 * case["rot"] + 4 + 4 * kv), "flops": rows * (heads + kv) * dim * 8}
    slots = sum(c + t for c, t in zip(held, new) if t)
    if case["op"] == "attn":
        pairs = sum(t * (c + (t + 1) / 2) for c, t in zip(held, new))
        out = 4 if case["out"] == "f32" else 2
        return {"bytes": slots * kv * dim * 4 + rows * heads * (dim * (2 + out) + 4), "flops": 4 * dim * heads * pairs}
    taken = [min(t, case["accepted"]) for t in new]
    if case["op"] == "score":
        pairs = sum(a * (c + t) for a, c, t in zip(taken, held, new))
        return {"bytes": slots * kv * (dim * 2 + 8) + sum(taken) * heads * (dim * 2 + 4), "flops": 2 * dim * heads * pairs}
    moved = seen = 0.0
    for c, t, a in zip(held, new, taken):
        n = c + a
        keep = min(n, case["budget"])
        seen += c + t
        moved += keep * (n - keep) / max(n, 1)  # the kept ones of the slots past the budget, if the weights say nothing about the slot
    return {"bytes": kv * (seen * 16 + moved * dim * 2 * 2 * 2), "flops": kv * seen * 8}


def drafts(case, rng):
    """The drafted tokens: for each sequence the parents of its nodes (-1: the
    last committed token) and which nodes are accepted, a path from the root."""
    parents, taken = [], []
    for t in lengths(case)[1]:
        a = min(t, case.get("accepted", 1))
        path = [0] + sorted(rng.sample(range(1, t), a - 1)) if t else []
        if not case["tree"]:
            path = list(range(a))
            parents.append([i - 1 for i in range(t)])
        else:
            up = [rng.randrange(-1, i) if i else -1 for i in range(t)]
            for above, node in zip([-1] + path, path):
                up[node] = above
            parents.append(up)
        taken.append(path)
    return parents, taken


def bits(rows, words):
    """Lists of set bits as packed 32-bit words [rows, words]."""
    x = np.zeros((len(rows), words * 32), dtype=np.uint8)
    for r, on in enumerate(rows):
        x[r, on] = 1
    return torch.from_numpy(np.packbits(x, axis=1, bitorder="little").view(np.int32).copy())


def prepare(case, seed):
    device = "cuda" if torch.cuda.is_available() else "cpu"
    rng = random.Random(seed)
    gen = torch.Generator(device=device).manual_seed(seed)
    held, new = lengths(case)
    n, heads, kv, dim, page = case["seqs"], case["heads"], case["kv"], case["dim"], case["page"]
    kind, rows = KINDS[case["kind"]], sum(new)

    def normal(*shape, by=1.0):
        return torch.randn(shape, generator=gen, device=device) * by

    def on(x, dtype=torch.int32):
        return torch.tensor(x, dtype=dtype).to(device)

    # the cache: pages of all sequences in no order, some of them spare
    most = max(c + t for c, t in zip(held, new))
    per = -(-most // page)
    pages = n * per + 3
    table = torch.randperm(pages, generator=gen, device=device)[: n * per].reshape(n, per).to(torch.int32)
    used = torch.arange(per, device=device)[None] * page < on([c + t for c, t in zip(held, new)])[:, None]
    table = torch.where(used, table, torch.full_like(table, -1)).contiguous()
    shape = (pages, page, kv, dim) if case["order"] == "token" else (pages, kv, page, dim)
    K, V = (torch.randn(shape, generator=gen, device=device, dtype=kind) for _ in range(2))
    if case["op"] in ("attn", "score"):  # memory that no token was written to holds anything
        idle = torch.ones(pages, page, dtype=torch.bool, device=device)
        slots = torch.arange(per * page, device=device)
        live = slots[None] < on([c + t for c, t in zip(held, new)])[:, None]
        b, at = torch.nonzero(live, as_tuple=True)
        idle[table[b, at // page].long(), at % page] = False
        spots = idle[:, :, None, None] if case["order"] == "token" else idle[:, None, :, None]
        K.masked_fill_(spots, float("nan"))
        V.masked_fill_(spots, float("nan"))
    if case["order"] == "head":
        K, V = K.transpose(1, 2), V.transpose(1, 2)
    cap = per * page

    parents, taken = drafts(case, rng)
    depth, up = [], []
    for p, c in zip(parents, held):
        d, seen = [], []
        for i, above in enumerate(p):
            d.append(d[above] + 1 if above >= 0 else 0)
            seen.append((seen[above] if above >= 0 else []) + [i] if case["tree"] else [])
        if case.get("blank") and seen:
            seen[0] = []
        depth += [c + x for x in d]
        up += seen
    words = max(1, -(-max(new) // 32))
    s = dict(case=case, K=K, V=V, table=table, held=on(held), indptr=on([0] + np.cumsum(new).tolist()), positions=on(depth),
             mask=bits(up, words).to(device) if case["tree"] else None, accept=bits(taken, words).to(device),
             nodes=max(new), ctx=max(held), scale=dim ** -0.5)
    if case["op"] == "rope":
        total = (heads + 2 * kv) * dim
        qkv = normal(rows, total).to(KINDS[case["src"]])  # the rows of one fused projection
        s["q"], s["k"], s["v"] = (x.unflatten(1, (-1, dim)) for x in qkv.split([heads * dim, kv * dim, kv * dim], dim=1))
        s["wq"], s["wk"] = (1 + normal(dim, by=0.1) if case["norm"] else None for _ in range(2))
        # angles of a context stretched fourfold
        turn = 10000.0 ** (-torch.arange(0, case["rot"], 2, dtype=torch.float64, device=device) / case["rot"]) / 4
        angle = torch.arange(most + 1, dtype=torch.float64, device=device)[:, None] * turn
        s["turns"] = torch.cat((angle.cos(), angle.sin()), 1).float().contiguous()
        s["pos"] = torch.full((n, kv, cap), -1, dtype=torch.int32, device=device)
    if case["op"] in ("attn", "score"):
        s["q"] = normal(rows, heads, dim, by=2.0).to(kind)
    if case["op"] == "score":
        s["lse"] = normal(rows, heads, by=0.3) + math.log(case["ctx"]) + 2.0
    if case["op"] in ("score", "evict"):
        # running sums: few tokens hold most of the weight, some none at all
        live = torch.arange(cap, device=device)[None] < s["held"][:, None]
        sums = torch.exp(normal(n, kv, cap, by=2.0)) * (torch.rand((n, kv, cap), generator=gen, device=device) > 0.05)
        s["score"] = torch.where(live[:, None], sums, torch.zeros_like(sums))
    if case["op"] == "evict":
        # earlier evictions left the tokens in no order of position
        order = torch.rand((n, kv, cap), generator=gen, device=device).masked_fill(~live[:, None], 2.0).argsort(-1).argsort(-1)
        spot = torch.arange(cap, device=device)[None] - s["held"][:, None]
        node = (s["indptr"][:-1, None] + spot).clamp(0, max(rows - 1, 0)).long()
        drafted = (spot >= 0) & (spot < (s["indptr"][1:] - s["indptr"][:-1])[:, None])
        s["pos"] = torch.where(live[:, None], order.to(torch.int32), torch.where(drafted, s["positions"][node], torch.full_like(node, -1, dtype=torch.int32))[:, None]).contiguous()
        s["ctx_out"], s["pos_out"], s["score_out"] = torch.zeros_like(s["held"]), torch.full_like(s["pos"], -1), torch.zeros_like(s["score"])
    if own:
        import xnor_popcount_gemm_amd as bnn

        s["cache"] = bnn.KVCache(K, V, table, pos=s.get("pos"), score=s.get("score"))
        if case["op"] == "attn":
            s["workspace"] = bnn.tree_attention_workspace(s["cache"], rows, heads, s["nodes"], s["ctx"])
        if case["op"] == "evict":
            s["workspace"] = bnn.cache_evict_workspace(s["cache"])
    return s


def run(s):
    return PLAIN[s["case"]["op"]](s) if not own else OWN[s["case"]["op"]](s)


# ---- the framework's calls


def own_rope(s):
    import xnor_popcount_gemm_amd as bnn

    q = bnn.qk_norm_rope(s["q"], s["k"], s["v"], s["cache"], s["indptr"], s["held"], s["positions"], s["turns"],
                         q_weight=s["wq"], k_weight=s["wk"], eps=EPS, interleaved=s["case"]["interleaved"])
    return {"q": q, "K": s["K"], "V": s["V"], "pos": s["pos"]}


def own_attn(s):
    import xnor_popcount_gemm_amd as bnn

    out, lse = bnn.tree_attention(s["q"], s["cache"], s["indptr"], s["held"], max_nodes=s["nodes"], max_ctx=s["ctx"], mask=s["mask"], scale=s["scale"],
                                  out_dtype=torch.float32 if s["case"]["out"] == "f32" else s["q"].dtype, workspace=s["workspace"])
    return {"out": out, "lse": lse}


def own_score(s):
    import xnor_popcount_gemm_amd as bnn

    out = torch.empty_like(s["score"])
    bnn.cache_score_add(s["q"], s["lse"], s["cache"], s["indptr"], s["held"], max_nodes=s["nodes"], max_ctx=s["ctx"], mask=s["mask"], accept=s["accept"],
                        scale=s["scale"], score_out=out)
    return {"score": out}


def own_evict(s):
    import xnor_popcount_gemm_amd as bnn

    bnn.cache_evict(s["cache"], s["indptr"], s["held"], budget=s["case"]["budget"], recent=s["case"]["recent"], accept=s["accept"], max_nodes=s["nodes"],
                    max_ctx=s["ctx"], ctx_out=s["ctx_out"], pos_out=s["pos_out"], score_out=s["score_out"], workspace=s["workspace"])
    return {"ctx": s["ctx_out"], "pos": s["pos_out"], "score": s["score_out"], "K": s["K"], "V": s["V"]}


OWN = {"rope": own_rope, "attn": own_attn, "score": own_score, "evict": own_evict}


# ---- the plain forms: elementary operations in 32 bits


def rows_of(s):
    """Of each drafted token its sequence and its place among that sequence's drafts."""
    at = torch.arange(s["positions"].numel(), device=s["indptr"].device, dtype=torch.int32)
    seq = torch.searchsorted(s["indptr"], at, right=True) - 1
    return seq, at.long() - s["indptr"][seq].long()


def plain_rope(s):
    case = s["case"]
    kind, rot, page = KINDS[case["kind"]], case["rot"], case["page"]
    c, d = s["turns"][s["positions"].long()][:, None].chunk(2, dim=-1)

    def turned(x, w):
        x = x.float()
        if w is not None:
            x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w
        y, rest = x[..., :rot], x[..., rot:]
        if case["interleaved"]:
            a, b = y[..., 0::2], y[..., 1::2]
            y = torch.stack((a * c - b * d, b * c + a * d), -1).flatten(-2)
        else:
            a, b = y.chunk(2, dim=-1)
            y = torch.cat((a * c - b * d, b * c + a * d), -1)
        return torch.cat((y, rest), -1).to(kind)

    seq, at = rows_of(s)
    slot = s["held"][seq].long() + at
    where = s["table"][seq, slot // page].long()
    s["K"][where, slot % page] = turned(s["k"], s["wk"])
    s["V"][where, slot % page] = s["v"].to(kind)
    s["pos"][seq, :, slot] = s["positions"][:, None].expand(-1, case["kv"])
    return {"q": turned(s["q"], s["wq"]), "K": s["K"], "V": s["V"], "pos": s["pos"]}


def gathered(s, cache):
    """The slots of all sequences [B, kv, slots, dim] in 32 bits, nothing in those that hold no token."""
    slots = s["nodes"] + s["ctx"]
    at = torch.arange(min(slots, s["table"].shape[1] * s["case"]["page"]), device=s["table"].device)
    page = s["table"].long()[:, at // s["case"]["page"]].clamp(min=0)
    live = at[None] < (s["held"] + s["indptr"][1:] - s["indptr"][:-1])[:, None]
    x = cache[page, at % s["case"]["page"]].float()
    return torch.where(live[:, :, None, None], x, 0.0).transpose(1, 2).contiguous()


def padded(s, x, fill=0.0):
    """Rows of all sequences [rows, ...] as [B, nodes, ...], and where they are."""
    n = s["indptr"].numel() - 1
    at = s["indptr"][:-1, None].long() + torch.arange(s["nodes"], device=x.device)
    there = at < s["indptr"][1:, None]
    y = x[at.clamp(max=x.shape[0] - 1)]
    return torch.where(there.reshape(n, s["nodes"], *[1] * (x.dim() - 1)), y, torch.full_like(y[:1, :1], fill)), there


def logits(s, K):
    """Scaled products of all rows with all slots [B, kv, nodes, group, slots] in 32 bits, and which slots each row sees [B, nodes, slots]."""
    case = s["case"]
    n, kv, slots, dim = K.shape
    q, there = padded(s, s["q"])
    group = case["heads"] // kv
    q = q.float().unflatten(2, (kv, group)).permute(0, 2, 1, 3, 4).reshape(n, kv, -1, dim)
    x = ((q * s["scale"]) @ K.transpose(2, 3)).unflatten(2, (s["nodes"], group))
    rel = (torch.arange(slots, device=K.device)[None] - s["held"][:, None])[:, None]
    new = (s["indptr"][1:] - s["indptr"][:-1])[:, None, None]
    if s["mask"] is None:
        drafted = rel <= torch.arange(s["nodes"], device=K.device)[:, None]
    else:
        words = padded(s, s["mask"], 0)[0]
        word = words.gather(2, (rel.clamp(0, 32 * words.shape[2] - 1) // 32).long().expand(-1, s["nodes"], -1))
        drafted = (word >> (rel.clamp(min=0) % 32)) & 1 != 0
    return x, ((rel < 0) | ((rel < new) & drafted)) & there[:, :, None]


def plain_attn(s):
    case = s["case"]
    V = gathered(s, s["V"])
    x, sees = logits(s, gathered(s, s["K"]))
    x = x.masked_fill(~sees[:, None, :, None], -math.inf)
    top = x.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    p = torch.exp(x - top)
    total = p.sum(-1, keepdim=True)
    n, kv, nodes, group, slots = p.shape
    out = (p.reshape(n, kv, nodes * group, slots) @ V).reshape(n, kv, nodes, group, -1) / torch.where(total == 0, 1.0, total)
    lse = (top + torch.log(total)).squeeze(-1)
    seq, at = rows_of(s)
    out = out.permute(0, 2, 1, 3, 4).flatten(2, 3)[seq, at]
    return {"out": out.to(torch.float32 if case["out"] == "f32" else KINDS[case["kind"]]), "lse": lse.permute(0, 2, 1, 3).flatten(2)[seq, at]}


def taken_rows(s):
    """Which rows are accepted [B, nodes]."""
    at = torch.arange(s["nodes"], device=s["accept"].device)
    return (s["accept"][:, at // 32] >> (at % 32)) & 1 != 0


def plain_score(s):
    x, sees = logits(s, gathered(s, s["K"]))
    n, kv, nodes, group, slots = x.shape
    lse = padded(s, s["lse"])[0].unflatten(2, (kv, group)).permute(0, 2, 1, 3)[..., None]
    sees = (sees & taken_rows(s)[:, :, None])[:, None, :, None] & (lse > -math.inf)
    p = torch.where(sees, torch.exp(x - lse), 0.0)
    out = s["score"].clone()
    out[:, :, :slots] += p.sum((2, 3))
    return {"score": out}


def plain_evict(s):
    case = s["case"]
    score, pos, held = s["score"], s["pos"].long(), s["held"].long()[:, None, None]
    n, kv, cap = score.shape
    new = (s["indptr"][1:] - s["indptr"][:-1]).long()[:, None, None]
    at = torch.arange(cap, device=score.device)[None, None]
    node = (at - held).clamp(0, s["nodes"] - 1)
    valid = (at < held) | ((at < held + new) & taken_rows(s)[torch.arange(n, device=score.device)[:, None, None], node])
    valid = valid.expand(n, kv, cap)
    keep = valid.sum(-1, keepdim=True).clamp(max=case["budget"])
    last = torch.where(valid, pos, -(1 << 40)).amax(-1, keepdim=True)
    # by weight, the lowest slot first among equals; recent tokens before all others, then those that hold no token last
    first = torch.where(torch.isnan(score), -math.inf, score).sort(dim=-1, descending=True, stable=True).indices
    rank = torch.where(valid, (pos > last - case["recent"]).long(), -1).gather(-1, first)
    first = first.gather(-1, rank.sort(dim=-1, descending=True, stable=True).indices)
    kept = torch.zeros_like(valid).scatter(-1, first, at < keep)
    # kept tokens past the budget go to the slots before it that are free, in order
    hole, mover = ~kept & (at < keep), kept & (at >= keep)
    count = torch.cumsum(mover, -1)
    source = torch.zeros_like(pos).scatter(-1, torch.where(mover, count - 1, cap - 1), at.expand(n, kv, cap) * mover)
    source = torch.where(hole, source.gather(-1, (torch.cumsum(hole, -1) - 1).clamp(min=0)), at)
    seen = at < held + new
    s["pos_out"].copy_(torch.where(at < keep, s["pos"].gather(-1, source), torch.where(seen, -1, s["pos_out"])))
    s["score_out"].copy_(torch.where(at < keep, score.gather(-1, source), torch.where(seen, 0.0, s["score_out"])))
    b, h, to = torch.nonzero(hole, as_tuple=True)
    come = source[b, h, to]
    table, page = s["table"].long(), case["page"]
    for cache in (s["K"], s["V"]):
        cache[table[b, to // page], to % page, h] = cache[table[b, come // page], come % page, h]
    s["ctx_out"].copy_(keep[:, 0, 0])
    return {"ctx": s["ctx_out"], "pos": s["pos_out"], "score": s["score_out"], "K": s["K"], "V": s["V"]}


PLAIN = {"rope": plain_rope, "attn": plain_attn, "score": plain_score, "evict": plain_evict}


# ---- the definitions in 64 bits


def unpacked(x):
    return np.unpackbits(np.ascontiguousarray(x.cpu().numpy()).view(np.uint8), axis=-1, bitorder="little").astype(bool)


def exact(case, seed):
    s = prepare(case, seed)
    return {"rope": exact_rope, "attn": exact_attn, "score": exact_score, "evict": exact_evict}[case["op"]](case, s)


def exact_rope(case, s):
    held, new = lengths(case)
    rot, half, page = case["rot"], case["rot"] // 2, case["page"]
    K, V, pos = s["K"].double(), s["V"].double(), s["pos"].clone()
    angles = s["turns"].double()[s["positions"].long()]
    cos, sin = angles[:, None, :half], angles[:, None, half:]
    i = torch.arange(half, device=K.device)
    first, second = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + half)

    def turned(x, w):
        x = x.double()
        if w is not None:
            x = x / (x.square().mean(-1, keepdim=True) + EPS).sqrt() * w.double()
        y = x.clone()
        y[..., first] = x[..., first] * cos - x[..., second] * sin
        y[..., second] = x[..., second] * cos + x[..., first] * sin
        return y

    k, row = turned(s["k"], s["wk"]), 0
    for b, (c, t) in enumerate(zip(held, new)):
        slot = torch.arange(c, c + t, device=K.device)
        where = s["table"][b].long()[slot // page]
        K[where, slot % page] = k[row:row + t]
        V[where, slot % page] = s["v"][row:row + t].double()
        pos[b][:, c:c + t] = s["positions"][row:row + t]
        row += t
    return {"q": turned(s["q"], s["wq"]), "K": K, "V": V, "pos": pos}


def one_sequence(case, s, b, c, t, row, cache):
    """The slots of sequence b [kv, slots, dim] in 64 bits."""
    slot = torch.arange(c + t, device=s["K"].device)
    return cache[s["table"][b].long()[slot // case["page"]], slot % case["page"]].double().permute(1, 0, 2)


def seen_by(case, s, b, c, t, row):
    """[t, c + t]: which slots each drafted token of sequence b sees."""
    sees = np.ones((t, c + t), dtype=bool)
    sees[:, c:] = np.tril(np.ones((t, t), dtype=bool)) if s["mask"] is None else unpacked(s["mask"][row:row + t])[:, :t]
    return torch.from_numpy(sees).to(s["K"].device)


def exact_attn(case, s):
    group = case["heads"] // case["kv"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=s["q"].device)
    lse = torch.full(s["q"].shape[:2], -math.inf, dtype=torch.float64, device=s["q"].device)
    row = 0
    for b, (c, t) in enumerate(zip(*lengths(case))):
        if t:
            k, v = (one_sequence(case, s, b, c, t, row, x) for x in (s["K"], s["V"]))
            sees = seen_by(case, s, b, c, t, row)
            for h in range(case["heads"]):
                x = (s["q"][row:row + t, h].double() @ k[h // group].T) * s["scale"]
                x[~sees] = -math.inf
                whole = torch.logsumexp(x, -1)
                lse[row:row + t, h] = whole
                p = torch.exp(x - whole[:, None])
                p[~sees] = 0.0
                out[row:row + t, h] = p @ v[h // group]
        row += t
    return {"out": out, "lse": lse}


def exact_score(case, s):
    group = case["heads"] // case["kv"]
    score, taken, row = s["score"].double(), unpacked(s["accept"]), 0
    for b, (c, t) in enumerate(zip(*lengths(case))):
        rows = [i for i in range(t) if taken[b, i]]
        if rows:
            k, sees = one_sequence(case, s, b, c, t, row, s["K"]), seen_by(case, s, b, c, t, row)[rows]
            for h in range(case["heads"]):
                x = (s["q"][row:row + t, h][rows].double() @ k[h // group].T) * s["scale"]
                p = torch.exp(x - s["lse"][row:row + t, h][rows].double()[:, None])
                score[b, h // group, : c + t] += torch.where(sees, p, 0.0).sum(0)
        row += t
    return {"score": score}


def exact_evict(case, s):
    held, new = lengths(case)
    taken, table, page = unpacked(s["accept"]), s["table"].cpu().numpy(), case["page"]
    score, pos = s["score"].cpu().numpy(), s["pos"].cpu().numpy()
    ctx, score_out, pos_out = np.zeros(len(held), np.int32), s["score_out"].cpu().numpy().astype(np.float64), s["pos_out"].cpu().numpy().copy()
    froms, tos = [], []
    for b, (c, t) in enumerate(zip(held, new)):
        valid = np.concatenate((np.arange(c), c + np.flatnonzero(taken[b, :t]))).astype(np.int64)
        keep = ctx[b] = min(len(valid), case["budget"])
        for h in range(case["kv"]):
            w, p = score[b, h, valid].astype(np.float64), pos[b, h, valid].astype(np.int64)
            recent = p > (p.max() if len(p) else 0) - case["recent"]
            stay = np.sort(valid[np.lexsort((valid, -w, ~recent))[:keep]])
            move, holes = stay[stay >= keep], np.setdiff1d(np.arange(keep), stay)
            source = np.arange(keep)
            source[holes] = move
            pos_out[b, h, :keep], pos_out[b, h, keep:c + t] = pos[b, h, source], -1
            score_out[b, h, :keep], score_out[b, h, keep:c + t] = score[b, h, source], 0
            for slots, into in ((move, froms), (holes, tos)):
                into.append(np.stack((table[b, slots // page], slots % page, np.full(len(slots), h)), 1))
    at, to = (torch.from_numpy(np.concatenate(x).astype(np.int64)).to(s["K"].device).unbind(1) for x in (froms, tos))
    caches = []
    for cache in (s["K"], s["V"]):
        new_cache = cache.double()
        new_cache[to] = cache[at].double()
        caches.append(new_cache)
    return {"ctx": torch.from_numpy(ctx), "pos": torch.from_numpy(pos_out), "score": torch.from_numpy(score_out), "K": caches[0], "V": caches[1]}
