"""The operators of a decoder's feed-forward half whose linear layers are 1-bit
ones on INT8 activations: what runs from the attention's output to the next
block's first projection.

  norm    experts' outputs joined, norm after the block, gate, residual, norm
          before the next block, INT8 quantization, in one pass
  route   the router: each token's experts and their weights, and the tokens
          in the order of their experts
  linear  binary or ternary matrices times INT8 rows, grouped by expert with
          ragged sizes (or one matrix), with bias, activation, product of a
          gate and residual in the epilogue
"""
import math
import random

import torch

own = False

KINDS = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZE = {"bf16": 2, "f16": 2, "f32": 4, "none": 0}
EPS = 1e-6
LEFT, LEFT_FLOAT = 77, 0.25  # what rows behind the last token hold before and after


def listed():
    norm = dict(op="norm", x="f32", branch="f32", parts=0, post="none", pre="rms", gate="none", y="none", q="rows", spare=0)
    route = dict(op="route", kind="f32", score="softmax", bias=False, renorm=True, spare=0)
    linear = dict(op="linear", weights="ternary", experts=8, top=2, gather=True, gated=False, act="none", bias=False, residual=False, out="f32", one_scale=True)
    return [
        # one token of one conversation, between attention and the feed-forward: latency; planes are what the one-row product reads
        dict(norm, name="norm_one_token", rows=1, dim=4096, q="planes"),
        # a padded batch, a width that is no multiple of anything: two experts' outputs joined, norms on both sides, a gate for each channel
        dict(norm, name="norm_batch_sandwich", rows=57, dim=1001, x="bf16", branch="bf16", parts=2, post="rms", pre="layer", gate="channel", y="bf16", spare=7),
        # prompts: the experts' outputs joined, the stream updated, the next block's rows and the router's input
        dict(norm, name="norm_prompts", rows=8192, dim=4096, parts=2, y="bf16"),
        # inside the feed-forward: norm of the hidden units and INT8 rows for the product down
        dict(norm, name="norm_hidden", rows=16384, dim=11008, x="none", branch="bf16"),
        # one token: latency
        dict(route, name="route_one_token", rows=1, experts=8, top=2),
        # a padded batch over fine-grained experts, chosen by a balanced score
        dict(route, name="route_batch", rows=200, experts=64, top=6, score="sigmoid", bias=True, spare=9),
        # prompts
        dict(route, name="route_prompts", rows=16384, experts=128, top=8, kind="bf16", renorm=False),
        # one token, the products up: two experts' matrices are read once
        dict(linear, name="linear_one_token", rows=1, dim=4096, width=11008, gated=True, act="silu", out="bf16"),
        # a decoding batch, the product down: all experts' matrices are read once, a few rows each
        dict(linear, name="linear_batch_down", rows=64, dim=11008, width=4096, gather=False),
        # many small experts, some without tokens, binary weights, odd sizes
        dict(linear, name="linear_fine_experts", rows=300, dim=1000, width=1013, weights="binary", experts=64, top=6, gated=True, act="relu2", one_scale=False, out="f16"),
        # prompts, the products up: bound by arithmetic
        dict(linear, name="linear_prompts", rows=8192, dim=4096, width=11008, gated=True, act="silu", out="bf16"),
        # a layer without experts: bias, activation and residual
        dict(linear, name="linear_plain_layer", rows=2000, dim=11008, width=4096, weights="binary", experts=1, top=1, gather=False, act="gelu", bias=True, residual=True,
             one_scale=False),
    ]


def spread(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(("norm", "norm", "route", "linear", "linear", "linear"))
    if op == "norm":
        c = dict(op=op, rows=spread(rng, 1, 16384), dim=spread(rng, 32, 12000))
        if rng.random() < 0.6:
            c["dim"] = -(-c["dim"] // 64) * 64
        c["x"] = rng.choice(("f32", "f32", "bf16", "f16", "none"))
        c["branch"] = rng.choice(("f32", "f32", "bf16", "f16", "none")) if c["x"] != "none" else rng.choice(("f32", "bf16"))
        c["parts"] = rng.choice((0, 0, 1, 2, 6)) if c["branch"] != "none" else 0
        c["post"] = rng.choice(("none", "none", "rms", "layer")) if c["branch"] != "none" else "none"
        c["gate"] = rng.choice(("none", "none", "channel", "row")) if c["branch"] != "none" else "none"
        c["pre"] = rng.choice(("rms", "rms", "layer", "none"))
        c["y"] = rng.choice(("none", "none", "f32", "bf16", "f16"))
        c["q"] = rng.choice(("rows", "rows", "planes" if c["rows"] <= 64 else "rows", "none" if c["y"] != "none" else "rows"))
        c["spare"] = rng.choice((0, 0, min(c["rows"] - 1, 5)))
        while work(c)["bytes"] > 8e8:
            c["rows"] = c["rows"] * 2 // 3
        return c
    if op == "route":
        c = dict(op=op, rows=spread(rng, 1, 16384), experts=spread(rng, 2, 256), kind=rng.choice(("f32", "f32", "bf16", "f16")), score=rng.choice(("softmax", "softmax", "sigmoid")),
                 bias=rng.random() < 0.3, renorm=rng.random() < 0.5)
        c["top"] = min(c["experts"], rng.choice((1, 2, 2, 4, 6, 8)))
        c["spare"] = rng.choice((0, 0, min(c["rows"] - 1, 5)))
        return c
    c = dict(op=op, rows=spread(rng, 1, 8192), dim=spread(rng, 100, 11008), width=spread(rng, 60, 11008), weights=rng.choice(("ternary", "ternary", "binary")))
    if rng.random() < 0.6:
        c["dim"], c["width"] = -(-c["dim"] // 64) * 64, -(-c["width"] // 64) * 64
    c["experts"] = rng.choice((1, 4, 8, 8, 16, spread(rng, 2, 64)))
    c["top"] = min(c["experts"], rng.choice((1, 2, 2, 4, 6)))
    c["gather"] = c["experts"] > 1 and rng.random() < 0.6
    c["gated"] = rng.random() < 0.5
    c["act"] = rng.choice(("silu", "gelu", "relu2", "relu", "gelu_tanh")) if c["gated"] else rng.choice(("none", "none", "gelu", "relu2"))
    c["bias"] = rng.random() < 0.3
    c["residual"] = not c["gated"] and rng.random() < 0.3
    c["out"] = rng.choice(("f32", "f32", "bf16", "f16"))
    c["one_scale"] = rng.random() < 0.6

    def dear(x):
        halves = 2 if x["gated"] else 1
        return work(x)["flops"] > 2.9e12 or x["experts"] * x["width"] * x["dim"] * halves > 7.2e8 or x["rows"] * x["top"] * max(x["dim"], x["width"]) > 1.8e8

    while dear(c):
        if c["experts"] * c["width"] * c["dim"] > 2e8 and c["experts"] > 4:
            c["experts"] = c["experts"] * 2 // 3
            c["top"] = min(c["top"], c["experts"])
        elif c["rows"] > 256:
            c["rows"] = c["rows"] * 2 // 3
        else:
            c["width"] = c["width"] * 2 // 3
    return c


def planes_ld(dim):
    return -(-dim // 128) * 4


def work(case):
    if case["op"] == "norm":
        n = case["rows"] - case["spare"]
        values = n * case["dim"]
        x = SIZE[case["x"]] * (2 if case["branch"] != "none" else 1)
        bytes_ = values * (x + SIZE[case["branch"]] * max(1, case["parts"]) + SIZE[case["y"]]) + 8 * n * case["parts"]
        bytes_ += {"rows": values + 4 * n, "planes": values + 8 * n + 32 * n * planes_ld(case["dim"]), "none": 0}[case["q"]]
        bytes_ += {"none": 0, "channel": 4 * case["dim"], "row": 4 * values}[case["gate"]] + 4 * case["dim"] * {"none": 0, "rms": 1, "layer": 2}[case["pre"]]
        return {"bytes": bytes_ + 4 * case["dim"] * {"none": 0, "rms": 1, "layer": 2}[case["post"]], "flops": 20 * values}
    if case["op"] == "route":
        n = case["rows"] - case["spare"]
        return {"bytes": n * (case["experts"] * SIZE[case["kind"]] + case["top"] * 16) + 4 * case["experts"], "flops": n * case["experts"] * 8}
    pairs, halves = case["rows"] * case["top"], 2 if case["gated"] else 1
    active = case["experts"] if case["experts"] == 1 else case["experts"] * (1 - (1 - case["top"] / case["experts"]) ** case["rows"])  # experts that a token chose, if they are chosen alike
    matrix = case["width"] * case["dim"] * halves / (8 if case["weights"] == "binary" else 4)
    rows = case["rows"] if case["gather"] else pairs
    return {"bytes": active * matrix + rows * (case["dim"] + 4) + pairs * case["width"] * SIZE[case["out"]] * (2 if case["residual"] else 1),
            "flops": 2.0 * pairs * case["width"] * case["dim"] * halves}


def chosen(case, gen, device):
    """Tokens sorted by their experts: where each expert's positions begin, the (token, choice) pair of each position, the longest run."""
    rows, experts, top = case["rows"], case["experts"], case["top"]
    favour = torch.randn(experts, generator=gen, device=device) * 0.5  # some experts are asked more often
    first = (torch.randn((rows, experts), generator=gen, device=device) + favour).topk(top, -1).indices.flatten()
    order = first.sort(stable=True).indices.to(torch.int32)
    count = torch.bincount(first, minlength=experts)
    offsets = torch.zeros(experts + 1, dtype=torch.int32, device=device)
    offsets[1:] = count.cumsum(0)
    return offsets, order, int(count.max())


def prepare(case, seed):
    device = "cuda" if torch.cuda.is_available() else "cpu"
    gen = torch.Generator(device=device).manual_seed(seed)

    def normal(*shape, by=1.0):
        return torch.randn(shape, generator=gen, device=device) * by

    s = dict(case=case)
    rows = case["rows"]
    if case["op"] == "norm":
        dim, parts = case["dim"], case["parts"]
        s["used"] = torch.tensor([rows - case["spare"]], dtype=torch.int32).to(device) if case["spare"] else None
        # a few channels of the stream are far larger than the others
        loud = 1 + 20.0 * (torch.rand(dim, generator=gen, device=device) < 0.01)
        s["x"] = (normal(rows, dim) * loud).to(KINDS[case["x"]]) if case["x"] != "none" else None
        if case["branch"] != "none":
            pairs = rows * max(1, parts)
            s["branch"] = normal(pairs, dim, by=0.7).to(KINDS[case["branch"]])
            if parts:
                s["place"] = torch.randperm(pairs, generator=gen, device=device).reshape(rows, parts).to(torch.int32)
                s["weight"] = torch.softmax(normal(rows, parts), -1)
        for side in ("post", "pre"):
            s[side + "_weight"] = 1 + normal(dim, by=0.1) if case[side] != "none" else None
            s[side + "_bias"] = normal(dim, by=0.1) if case[side] == "layer" else None
        s["gate"] = {"none": None, "channel": normal(dim, by=0.3) if case["gate"] == "channel" else None, "row": normal(rows, dim, by=0.3) if case["gate"] == "row" else None}[case["gate"]]
        s["scales"] = (1.0, 0.5 if case["gate"] == "none" else 1.0)
        out = {}
        if case["x"] != "none" and case["branch"] != "none":
            out["x"] = torch.full((rows, dim), LEFT_FLOAT, dtype=KINDS[case["x"]], device=device)
        if case["y"] != "none":
            out["y"] = torch.full((rows, dim), LEFT_FLOAT, dtype=KINDS[case["y"]], device=device)
        if case["q"] != "none":
            out["Xq"] = torch.full((rows, -(-dim // 16) * 16), LEFT, dtype=torch.int8, device=device)[:, :dim]
            out["xscale"] = torch.full((rows,), LEFT_FLOAT, dtype=torch.float32, device=device)
        if case["q"] == "planes":
            out["Xb"] = torch.full((rows, 8, planes_ld(dim)), LEFT, dtype=torch.int32, device=device)
            out["xsum"] = torch.full((rows,), LEFT, dtype=torch.int32, device=device)
        s["out"] = out
    elif case["op"] == "route":
        experts, top = case["experts"], case["top"]
        s["used"] = torch.tensor([rows - case["spare"]], dtype=torch.int32).to(device) if case["spare"] else None
        logits = normal(rows, experts, by=1.5) + normal(experts, by=0.5)
        logits[torch.rand(logits.shape, generator=gen, device=device) < 0.01] = -math.inf  # experts that a token may not use
        if rows > 20:
            logits[rows // 3] = -math.inf  # a token that may use none
        s["logits"] = logits.to(KINDS[case["kind"]])
        s["bias"] = normal(experts, by=0.1) if case["bias"] else None
        whole = dict(dtype=torch.int32, device=device)
        s["out"] = {"expert": torch.full((rows, top), LEFT, **whole), "weight": torch.full((rows, top), LEFT_FLOAT, device=device),
                    "offsets": torch.full((experts + 1,), LEFT, **whole), "order": torch.full((rows * top,), LEFT, **whole), "place": torch.full((rows, top), LEFT, **whole)}
        if own:
            import xnor_popcount_gemm_amd as bnn

            s["workspace"] = bnn.expert_route_workspace(rows, experts, top, device=device)
    else:
        dim, width, experts = case["dim"], case["width"], case["experts"]
        s["offsets"] = s["order"] = None
        pairs = s["most"] = rows
        if experts > 1:
            s["offsets"], s["order"], s["most"] = chosen(case, gen, device)
            pairs = rows * case["top"]
        s["pairs"] = pairs
        n = rows if case["gather"] or experts == 1 else pairs
        s["Xq"] = torch.full((n, -(-dim // 16) * 16), LEFT, dtype=torch.int8, device=device)[:, :dim]
        s["Xq"].copy_(normal(n, dim, by=32.0).round().clamp(-127, 127))
        s["xscale"] = 0.01 + 0.02 * torch.rand(n, generator=gen, device=device)
        s["weights"] = []
        for _ in range(2 if case["gated"] else 1):
            t = torch.randint(-1 if case["weights"] == "ternary" else 0, 2, (experts, width, dim), generator=gen, device=device, dtype=torch.int8)
            if case["weights"] == "binary":
                t = 2 * t - 1
            by = 1.2 / (0.6 * math.sqrt(dim))
            alpha = by * (0.8 + 0.4 * torch.rand(experts if case["one_scale"] else (experts, width), generator=gen, device=device))
            s["weights"].append(dict(t=t, alpha=alpha, bias=normal(experts, width, by=0.2) if case["bias"] else None))
        s["residual"] = normal(pairs, width).to(KINDS[case["out"]]) if case["residual"] else None
        if own:
            import xnor_popcount_gemm_amd as bnn

            for w in s["weights"]:
                if case["weights"] == "ternary":
                    planes = [bnn.pack_weights_ternary(m.float(), delta=0.5)[:2] for m in w["t"]]
                    sign, nonzero = (torch.stack(p) for p in zip(*planes))
                else:
                    sign, nonzero = torch.stack([bnn.pack_weights(m.float(), alpha=False)[0] for m in w["t"]]), None
                w["own"] = bnn.ExpertWeights(sign, dim, Zp=nonzero, alpha=w["alpha"], bias=w["bias"])
    return s


def run(s):
    return PLAIN[s["case"]["op"]](s) if not own else OWN[s["case"]["op"]](s)


# ---- the framework's calls


def own_norm(s):
    import xnor_popcount_gemm_amd as bnn

    c = s["case"]
    return bnn.block_norm(s["x"], s.get("branch"), place=s.get("place"), weight=s.get("weight"), post=c["post"], post_weight=s["post_weight"], post_bias=s["post_bias"],
                          gate=s["gate"], x_scale=s["scales"][0], branch_scale=s["scales"][1], pre=c["pre"], pre_weight=s["pre_weight"], pre_bias=s["pre_bias"], eps=EPS,
                          used=s["used"], out=s["out"])


def own_route(s):
    import xnor_popcount_gemm_amd as bnn

    c = s["case"]
    return bnn.expert_route(s["logits"], c["top"], score=c["score"], bias=s["bias"], renorm=c["renorm"], scale=1.0, used=s["used"], out=s["out"], workspace=s["workspace"])


def own_linear(s):
    import xnor_popcount_gemm_amd as bnn

    c, w = s["case"], s["weights"]
    return bnn.expert_linear(s["Xq"], w[0]["own"], xscale=s["xscale"], offsets=s["offsets"], order=s["order"] if c["gather"] else None, per_row=c["top"],
                             up=w[1]["own"] if c["gated"] else None, act=c["act"], residual=s["residual"], out_dtype=KINDS[c["out"]])


OWN = {"norm": own_norm, "route": own_route, "linear": own_linear}


# ---- the plain forms: elementary operations


def kept(s, name, new):
    """`new`, but in the rows behind the last token what was there."""
    old = s["out"][name]
    if s["used"] is None:
        return new
    at = torch.arange(old.shape[0], device=old.device).reshape(-1, *[1] * (old.dim() - 1))
    return torch.where(at < s["used"], new, old)


def normed(x, kind, weight, bias):
    if kind == "none":
        return x
    if kind == "layer":
        x = x - x.mean(-1, keepdim=True)
    y = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * weight
    return y if bias is None else y + bias


def plain_norm(s):
    c = s["case"]
    # the codes lie next to a border between two of them for some of millions of values: 64 bits up to the rounding to 32
    wide = torch.float64 if c["q"] != "none" else torch.float32
    x = s["x"].to(wide) * s["scales"][0] if s["x"] is not None else None
    out = {}
    if c["branch"] != "none":
        b = s["branch"].to(wide)
        if c["parts"]:
            b = (b[s["place"].long()] * s["weight"][:, :, None]).sum(1)
        b = normed(b, c["post"], s["post_weight"], s["post_bias"])
        if s["gate"] is not None:
            b = b * s["gate"]
        b = b * s["scales"][1]
        if x is None:
            x = b
        else:
            x = (x + b).to(KINDS[c["x"]])
            out["x"] = kept(s, "x", x)
            x = x.to(wide)
    y = normed(x, c["pre"], s["pre_weight"], s["pre_bias"])
    if c["y"] != "none":
        out["y"] = kept(s, "y", y.to(KINDS[c["y"]]))
    if c["q"] != "none":
        y = y.float()
        most = y.abs().amax(-1, keepdim=True)
        code = torch.round(y * torch.where(most > 0, 127.0 / most, 0.0)).clamp(-127, 127).to(torch.int8)
        out["Xq"] = kept(s, "Xq", code)
        out["xscale"] = kept(s, "xscale", (most / 127.0).squeeze(-1))
    if c["q"] == "planes":
        whole = code.to(torch.int64) & 255
        out["xsum"] = kept(s, "xsum", code.sum(-1, dtype=torch.int32))
        ld = planes_ld(c["dim"])
        whole = torch.nn.functional.pad(whole, (0, 32 * ld - c["dim"])).reshape(-1, 1, ld, 32)
        bit = (whole >> torch.arange(8, device=whole.device).reshape(8, 1, 1)) & 1
        words = (bit << torch.arange(32, device=whole.device)).sum(-1)
        out["Xb"] = kept(s, "Xb", torch.where(words >= 1 << 31, words - (1 << 32), words).to(torch.int32))
    return out


def plain_route(s):
    c = s["case"]
    rows, experts, top = c["rows"], c["experts"], c["top"]
    logits = s["logits"].float()

    def scores(x):
        if c["score"] == "sigmoid":
            return 1 / (1 + torch.exp(-x))
        most = x.amax(-1, keepdim=True)
        e = torch.exp(x - torch.where(most == -math.inf, 0.0, most))
        total = e.sum(-1, keepdim=True)
        return e / torch.where(total == 0, 1.0, total)

    key = logits
    if s["bias"] is not None:  # two experts' scores can be next to each other
        key = torch.where(logits == -math.inf, -math.inf, scores(logits.double()) + s["bias"])
    key, first = (x[:, :top] for x in key.sort(dim=-1, descending=True, stable=True))
    row = torch.arange(rows, device=logits.device)
    live = key > -math.inf
    if s["used"] is not None:
        live = live & (row < s["used"])[:, None]
    weight = torch.where(live, scores(logits).gather(-1, first), 0.0)
    if c["renorm"]:
        total = weight.sum(-1, keepdim=True)
        weight = weight / torch.where(total == 0, 1.0, total)
    expert = torch.where(live, first, experts)
    order = expert.flatten().sort(stable=True).indices
    at = torch.arange(rows * top, device=logits.device)
    place = torch.empty_like(order).scatter_(0, order, at).reshape(rows, top)
    count = torch.zeros(experts + 1, dtype=torch.int64, device=logits.device).scatter_add_(0, expert.flatten(), torch.ones_like(at))
    end = count[:experts].cumsum(0)
    offsets = torch.cat((torch.zeros_like(end[:1]), end)).to(torch.int32)
    return {"expert": kept(s, "expert", torch.where(live, first, -1).to(torch.int32)), "weight": kept(s, "weight", weight), "offsets": offsets,
            "order": torch.where(at < end[-1], order.to(torch.int32), s["out"]["order"]), "place": kept(s, "place", torch.where(live, place, -1).to(torch.int32))}


def activated(z, act):
    if act == "relu":
        return torch.clamp(z, min=0)
    if act == "relu2":
        return torch.clamp(z, min=0) ** 2
    if act == "silu":
        return z / (1 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z / math.sqrt(2.0)))
    if act == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z ** 3)))
    return z


def plain_linear(s):
    c = s["case"]
    device = s["Xq"].device
    offsets = s["offsets"] if s["offsets"] is not None else torch.tensor([0, s["pairs"]], dtype=torch.int32, device=device)
    position = torch.arange(s["pairs"], device=device, dtype=torch.int32)
    expert = torch.searchsorted(offsets[1:], position, right=True)
    row = (s["order"] // c["top"]).long() if c["gather"] else position.long()
    few = s["pairs"] < c["experts"]  # then the matrices of the experts asked for, otherwise each expert's rows side by side, up to the most that one has
    slot = torch.arange(s["most"], device=device) + offsets[:-1, None]
    X = s["Xq"][row[:, None] if few else row[slot.clamp(max=s["pairs"] - 1).long()]].float()  # sums of products stay whole numbers below 2^24
    z = []
    for w in s["weights"]:
        D = torch.matmul(X, (w["t"][expert] if few else w["t"]).float().transpose(1, 2))
        D = D[:, 0] if few else D[expert, position.long() - offsets[expert].long()]
        alpha = w["alpha"][expert][:, None] if c["one_scale"] else w["alpha"][expert]
        y = alpha * D * s["xscale"][row][:, None]
        z.append(y if w["bias"] is None else y + w["bias"][expert])
    y = activated(z[0], c["act"])
    if c["gated"]:
        y = y * z[1]
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return y.to(KINDS[c["out"]])


PLAIN = {"norm": plain_norm, "route": plain_route, "linear": plain_linear}


# ---- the definitions in 64 bits


def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": exact_norm, "route": exact_route, "linear": exact_linear}[case["op"]](case, s)


def exact_norm(case, s):
    used = case["rows"] - case["spare"]

    def whole(name, rows):
        out = s["out"][name].double()
        out[:used] = rows
        return out

    def norm(v, kind, side):
        if kind == "none":
            return v
        if kind == "layer":
            v = v - v.sum(1, keepdim=True) / v.shape[1]
        v = v / (v.square().sum(1, keepdim=True) / v.shape[1] + EPS).sqrt() * s[side + "_weight"].double()
        return v + s[side + "_bias"].double() if s[side + "_bias"] is not None else v

    stream = None if s["x"] is None else s["x"][:used].double() * s["scales"][0]
    out = {}
    if case["branch"] != "none":
        if case["parts"]:
            b = torch.zeros((used, case["dim"]), dtype=torch.float64, device=s["branch"].device)
            for j in range(case["parts"]):
                b += s["weight"][:used, j, None].double() * s["branch"][s["place"][:used, j].long()].double()
        else:
            b = s["branch"][:used].double()
        b = norm(b, case["post"], "post")
        if s["gate"] is not None:
            b = b * (s["gate"] if case["gate"] == "channel" else s["gate"][:used]).double()
        b = b * s["scales"][1]
        if stream is None:
            stream = b
        else:
            stream = stream + b
            out["x"] = whole("x", stream)
            stream = stream.to(KINDS[case["x"]]).double()  # the norm reads the stream as it is stored
    y = norm(stream, case["pre"], "pre")
    if case["y"] != "none":
        out["y"] = whole("y", y)
    if case["q"] != "none":
        out["xscale"] = whole("xscale", y.abs().amax(1) / 127)
        out["Xq"] = None  # whole numbers
    if case["q"] == "planes":
        out["Xb"] = out["xsum"] = None
    return out


def exact_route(case, s):
    used = case["rows"] - case["spare"]
    logits = s["logits"][:used].double()
    if case["score"] == "sigmoid":
        score = torch.special.expit(logits)
    else:
        score = torch.nan_to_num(torch.softmax(logits, -1), nan=0.0)
    key = logits if s["bias"] is None else torch.where(torch.isinf(logits), logits, score + s["bias"].double())
    order = torch.argsort(-key, dim=-1, stable=True)[:, : case["top"]]
    w = score.gather(1, order) * (key.gather(1, order) > -math.inf)
    if case["renorm"]:
        w = w / w.sum(1, keepdim=True).clamp(min=1e-300)
    weight = s["out"]["weight"].double()
    weight[:used] = w
    return {"expert": None, "weight": weight, "offsets": None, "order": None, "place": None}


def exact_linear(case, s):
    pairs = s["pairs"]
    out = torch.empty((pairs, case["width"]), dtype=torch.float64, device=s["Xq"].device)
    ends = [0, pairs] if s["offsets"] is None else s["offsets"].tolist()
    for e in range(case["experts"]):
        lo, hi = ends[e], ends[e + 1]
        rows = s["order"][lo:hi].long() // case["top"] if case["gather"] else torch.arange(lo, hi, device=out.device)
        x = s["Xq"][rows].double()
        z = []
        for w in s["weights"]:
            y = (x @ w["t"][e].double().T) * w["alpha"][e].double() * s["xscale"][rows, None].double()
            z.append(y if w["bias"] is None else y + w["bias"][e].double())
        g = z[0]
        y = {"none": lambda: g, "relu": lambda: g.clamp(min=0), "relu2": lambda: g.clamp(min=0).square(), "silu": lambda: g * torch.special.expit(g),
             "gelu": lambda: g * torch.special.ndtr(g), "gelu_tanh": lambda: g * torch.special.expit(math.sqrt(8 / math.pi) * (g + 0.044715 * g ** 3))}[case["act"]]()
        if case["gated"]:
            y = y * z[1]
        out[lo:hi] = y if s["residual"] is None else y + s["residual"][lo:hi].double()
    return out
