"""The feed-forward calls on the GPU against their definitions in 64 bits."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import ffn_ref as ref
from gpu_util import banner, require_gpu

pytestmark = pytest.mark.gpu
KINDS = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
LEFT = 77


@pytest.fixture(scope="module")
def bnn():
    require_gpu()
    import xnor_popcount_gemm_amd as m
    m.lib()
    return m


def near(got, want, bound, dtype, what):
    """|got - want| <= bound + half a step of dtype; infinities and NaN alike."""
    g, w = ref.f64(got), np.asarray(want, dtype=np.float64)
    with np.errstate(all="ignore"):
        off = np.abs(g - w) <= bound + ref.U[dtype] * np.abs(w) * 1.01 + ref.TINY[dtype]
        big = np.abs(w) > torch.finfo(dtype).max    # past the type's range: infinite
        off |= (g == w) | (np.isnan(g) & np.isnan(w)) | (big & (g == np.where(w > 0, np.inf, -np.inf)))
    assert off.all(), f"{what}: {int((~off).sum())} of {off.size} off, first at {np.argwhere(~off)[0]}: {g[~off][0]} for {w[~off][0]}"


def make(rng, shape, dtype=torch.float32, by=1.0):
    return torch.from_numpy((rng.standard_normal(shape) * by).astype(np.float32)).to(dtype).cuda()


def strided(t, pad):
    """The same matrix with rows `pad` values further apart."""
    if t is None or not pad:
        return t
    big = torch.empty((t.shape[0], t.shape[1] + pad), dtype=t.dtype, device=t.device)
    big[:, : t.shape[1]] = t
    return big[:, : t.shape[1]]


# ---- block_norm


def check_norm(bnn, x, branch, *, used=None, y="f32", q=True, pad=0, out_x=True, what="", **kw):
    """One call with all outputs, into buffers that hold LEFT, against the definition."""
    M = x.shape[0] if x is not None else kw["place"].shape[0] if kw.get("place") is not None else branch.shape[0]
    D = (x if x is not None else branch).shape[1]
    out = {"y": strided(torch.full((M, D), LEFT, dtype=KINDS[y], device="cuda"), pad)}
    if x is not None and branch is not None and out_x:
        out["x"] = strided(torch.full((M, D), LEFT, dtype=x.dtype, device="cuda"), pad)
    if q:
        out["Xq"] = torch.full((M, bnn.i8_ld(D) + 16 * (pad > 0)), LEFT, dtype=torch.int8, device="cuda")[:, :D]
        out["Xb"] = torch.full((M, 8, bnn.padded_ld(D) + 4 * (pad > 0)), LEFT, dtype=torch.int32, device="cuda")
        out["xsum"] = torch.full((M,), LEFT, dtype=torch.int32, device="cuda")
        out["xscale"] = torch.full((M,), LEFT, dtype=torch.float32, device="cuda")
    got = bnn.block_norm(strided(x, pad), strided(branch, pad), used=None if used is None else torch.tensor([used], dtype=torch.int32).cuda(), out=out, **kw)
    torch.cuda.synchronize()
    assert got is out
    s, stored, v = ref.block_norm(x, branch, store="x" in out, **kw)
    n = M if used is None else max(0, min(M, used))
    for t in out.values():
        assert (t[n:] == LEFT).all(), f"{what}: rows behind the last one were written"
    if "x" in out:
        near(out["x"][:n], s[:n], ref.E32 * np.abs(s[:n]), x.dtype, what + " x")
        if not np.array_equal(ref.f64(out["x"][:n]), stored[:n], equal_nan=True):   # next to a border of the type: y follows the stored one
            stored = np.concatenate((ref.f64(out["x"][:n]), stored[n:]))
            v = ref.norm(stored, kw.get("pre", "rms"), kw.get("pre_weight"), kw.get("pre_bias"), kw.get("eps", 1e-6))
    # 64-bit rows, 2^-40 of the largest term of a sum for their order, rounded to 32 bits and to the output's type
    with np.errstate(all="ignore"):
        most = np.nanmax(np.where(np.isinf(v), 0, np.abs(v)), -1, initial=0, keepdims=True)[:n]
    near(out["y"][:n], v[:n], ref.E32 * np.abs(v[:n]) + 2.0 ** -40 * most, KINDS[y], what + " y")
    if q and n:
        # the codes are those of the fp32 rows; y in fp32 shows them
        rows = ref.f64(out["y"][:n]).astype(np.float32) if y == "f32" else v[:n].astype(np.float32)
        code, scale, total = ref.quantized(rows)
        differ = (out["Xq"][:n].cpu().numpy() != code).mean()
        if y == "f32":
            assert differ == 0, f"{what}: {differ} of the codes differ"
            np.testing.assert_array_equal(out["xscale"][:n].cpu().numpy(), scale)
        else:
            assert differ <= 1e-3 and np.abs(out["Xq"][:n].cpu().numpy().astype(int) - code).max() <= 1
        code = out["Xq"][:n].contiguous().cpu().numpy()
        np.testing.assert_array_equal(out["xsum"][:n].cpu().numpy(), code.astype(np.int32).sum(-1))
        np.testing.assert_array_equal(out["Xb"][:n].cpu().numpy(), ref.planes(code, out["Xb"].shape[2]))
    return out


@pytest.mark.parametrize("D", [1, 3, 4, 31, 64, 100, 128, 255, 256, 500, 513, 1000, 1024, 1025, 2048, 2051, 4096, 4100, 5000, 8192, 8195, 11008, 16381, 16384])
def test_norm_widths(bnn, D):
    rng = np.random.default_rng(D)
    banner(f"norm D={D}")
    w = make(rng, D, by=0.1) + 1
    check_norm(bnn, make(rng, (5, D)), make(rng, (5, D)), pre_weight=w, what=f"D={D}")
    check_norm(bnn, make(rng, (3, D), torch.bfloat16), make(rng, (3, D), torch.float16), pad=1 + D % 4, pre="layer", post="rms", what=f"D={D} strided")


@pytest.mark.parametrize("kx", ["f32", "bf16", "f16", None])
@pytest.mark.parametrize("kb", ["f32", "bf16", "f16", None])
@pytest.mark.parametrize("y", ["f32", "bf16", "f16"])
def test_norm_types(bnn, kx, kb, y):
    if kx is None and kb is None:
        return
    rng = np.random.default_rng(1)
    banner(f"norm types {kx} {kb} {y}")
    for D in (96, 1001):
        x = make(rng, (6, D), KINDS[kx], 3.0) if kx else None
        b = make(rng, (6, D), KINDS[kb]) if kb else None
        check_norm(bnn, x, b, y=y, what=f"{kx} {kb} {y} {D}")


@pytest.mark.parametrize("post", ["none", "rms", "layer"])
@pytest.mark.parametrize("pre", ["none", "rms", "layer"])
@pytest.mark.parametrize("gate", [None, "channel", "row"])
@pytest.mark.parametrize("D", [200, 1500])
def test_norm_sandwich(bnn, post, pre, gate, D):
    rng = np.random.default_rng(2)
    M = 7
    banner(f"norm {post} {pre} {gate} {D}")
    kw = dict(post=post, pre=pre, x_scale=0.75, branch_scale=-1.5, eps=1e-5)
    if post != "none":
        kw |= dict(post_weight=1 + make(rng, D, by=0.2), post_bias=make(rng, D, by=0.2))
    if pre != "none":
        kw |= dict(pre_weight=1 + make(rng, D, by=0.2), pre_bias=make(rng, D, by=0.2))
    if gate:
        kw["gate"] = make(rng, D) if gate == "channel" else make(rng, (M, D))
    check_norm(bnn, make(rng, (M, D)), make(rng, (M, D)), what=f"{post} {pre} {gate}", **kw)


@pytest.mark.parametrize("parts", [1, 2, 3, 8, 64])
@pytest.mark.parametrize("weighted", [True, False])
def test_norm_joins_experts(bnn, parts, weighted):
    """Rows of the branch by place: some twice, some nowhere (-1, past the end)."""
    rng = np.random.default_rng(parts)
    M, D, R = 9, 333, 20
    banner(f"norm parts {parts}")
    place = rng.integers(-1, R + 2, (M, parts)).astype(np.int32)
    place[2] = -1                    # a row that no expert has
    place[3] = 4                     # the same row of the branch again and again
    place[4, 0], place[5, 0] = 2 ** 31 - 1, -2 ** 31
    kw = dict(place=torch.from_numpy(place).cuda())
    if weighted:
        kw["weight"] = make(rng, (M, parts))
    for x in (make(rng, (M, D)), None):
        check_norm(bnn, x, make(rng, (R, D)), what=f"parts {parts}", **kw)


@pytest.mark.parametrize("used", [-3, 0, 1, 4, 6, 7, 100])
@pytest.mark.parametrize("D", [60, 700])
def test_norm_padded_batch(bnn, used, D):
    rng = np.random.default_rng(3)
    banner(f"norm used {used}")
    check_norm(bnn, make(rng, (6, D)), make(rng, (6, D)), used=used, what=f"used {used}")


@pytest.mark.parametrize("D", [70, 1200])
def test_norm_values(bnn, D):
    """Zero rows, infinities, NaN, large and tiny values; eps 0."""
    rng = np.random.default_rng(4)
    x = rng.standard_normal((9, D)).astype(np.float32)
    x[0] = 0
    x[1, 5], x[2, 7], x[3, 3], x[3, 60] = np.inf, np.nan, np.inf, -np.inf
    x[4] *= 1e30
    x[5] *= 1e-30
    x[6] = 3.0
    x[7, 0] = 1e38
    banner(f"norm values {D}")
    for pre in ("none", "rms", "layer"):
        for eps in (1e-6, 0.0):
            check_norm(bnn, torch.from_numpy(x).cuda(), None, pre=pre, eps=eps, what=f"{pre} {eps}")


def test_norm_in_place(bnn):
    rng = np.random.default_rng(5)
    banner("norm in place")
    for D in (64, 1024, 5000):
        x, b = make(rng, (4, D)), make(rng, (4, D))
        want = bnn.block_norm(x, b, y_dtype=torch.float32)
        same = x.clone()
        got = bnn.block_norm(same, b, out={"x": same, "y": torch.empty_like(x)})
        torch.cuda.synchronize()
        assert torch.equal(got["x"], want["x"]) and torch.equal(got["y"], want["y"]) and got["x"] is same


def test_norm_rows_like_the_quantizers(bnn):
    """Codes and scales as quantize_act_i8 gives them for the same fp32 rows, but for codes next to a border (its factor
    127 / amax has one rounding, a reciprocal times 127 two: products apart by 127 * 2 * 2^-23 at most)."""
    rng = np.random.default_rng(6)
    banner("norm against the quantizer")
    for D in (100, 1000, 4096):
        x = make(rng, (3, D))
        a = bnn.block_norm(x, pre="rms", y_dtype=torch.float32, planes=True)
        b = bnn.quantize_act_i8(a["y"])
        torch.cuda.synchronize()
        assert torch.equal(a["xscale"], b["xscale"])
        at = ref.f64(a["y"]) * 127 / np.abs(ref.f64(a["y"])).max(-1, keepdims=True)
        border = np.abs(at - np.floor(at) - 0.5) < 127 * 2.0 ** -21
        assert ((a["Xq"] == b["Xq"]).cpu().numpy() | border).all() and (a["Xq"].int() - b["Xq"].int()).abs().max() <= 1


def test_norm_many_rows(bnn):
    rng = np.random.default_rng(7)
    banner("norm 70000 rows")
    x = make(rng, (70000, 40), torch.bfloat16)
    got = bnn.block_norm(x, x, y_dtype=torch.float32)
    torch.cuda.synchronize()
    _, stored, v = ref.block_norm(x, x)
    np.testing.assert_array_equal(ref.f64(got["x"]), stored)
    near(got["y"], v, ref.E32 * np.abs(v) + 1e-9, torch.float32, "y")


# ---- expert_route


def check_route(bnn, logits, top, *, used=None, what="", **kw):
    rows, E = logits.shape
    whole = dict(dtype=torch.int32, device="cuda")
    out = {"expert": torch.full((rows, top), -9, **whole), "weight": torch.full((rows, top), -9.0, device="cuda"), "offsets": torch.full((E + 1,), -9, **whole),
           "order": torch.full((rows * top,), -9, **whole), "place": torch.full((rows, top), -9, **whole)}
    got = bnn.expert_route(logits, top, used=None if used is None else torch.tensor([used], dtype=torch.int32).cuda(), out=out, **kw)
    torch.cuda.synchronize()
    assert got is out
    expert, weight, offsets, order, place = ref.expert_route(logits, top, used=used, **kw)
    np.testing.assert_array_equal(out["expert"].cpu().numpy(), expert, err_msg=what)
    np.testing.assert_array_equal(out["offsets"].cpu().numpy(), offsets, err_msg=what)
    np.testing.assert_array_equal(out["place"].cpu().numpy(), place, err_msg=what)
    o = out["order"].cpu().numpy()
    np.testing.assert_array_equal(o[: len(order)], order, err_msg=what)
    assert (o[len(order):] == -9).all(), what
    # exponentials of rounded differences (|l - max| E32 each, 2 ulp), a sum of E terms in any order, quotients
    x = np.abs(np.nan_to_num(ref.f64(logits), nan=0, posinf=0, neginf=0)).max(initial=0)
    bound = (2 * x + E + 12) * ref.E32 * (2 if kw.get("renorm") else 1)
    near(out["weight"], weight, bound * np.abs(weight), torch.float32, what)


@pytest.mark.parametrize("rows", [0, 1, 2, 63, 64, 65, 200, 1000])
@pytest.mark.parametrize("E,top", [(1, 1), (2, 1), (8, 2), (60, 6), (64, 64), (65, 3), (128, 8), (200, 5), (257, 9), (1024, 64)])
def test_route_sizes(bnn, rows, E, top):
    rng = np.random.default_rng(rows * 1000 + E)
    if rows * E > 300000:
        rows = 100
    banner(f"route {rows} {E} {top}")
    check_route(bnn, make(rng, (rows, E)), top, renorm=E % 2 == 0, what=f"{rows} {E} {top}")


@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("renorm", [False, True])
def test_route_kinds(bnn, kind, score, bias, renorm):
    rng = np.random.default_rng(8)
    banner(f"route {kind} {score} {bias} {renorm}")
    for rows, E, top in ((40, 30, 4), (300, 130, 7)):
        l = strided(make(rng, (rows, E), KINDS[kind], 2.0), 5)
        check_route(bnn, l, top, score=score, bias=make(rng, E, by=0.3) if bias else None, renorm=renorm, scale=2.5, what=f"{kind} {score}")


@pytest.mark.parametrize("rows", [30, 500])
def test_route_ties_and_masks(bnn, rows):
    rng = np.random.default_rng(9)
    E, top = 70, 6
    l = np.round(rng.standard_normal((rows, E)) * 2) / 2          # many equal logits
    l[0] = 1.0                                                    # all equal
    l[1] = -np.inf                                                # no expert at all
    l[2] = -np.inf
    l[2, 33] = 0.5                                                # only one
    l[3, ::2] = np.nan
    l[4] = np.nan
    l[5, :10] = [0.0, -0.0] * 5                                   # zeros of both signs are equal
    l[5, 10:] = -5
    l[6] = -1e30
    l[7, 3] = 3e38
    banner(f"route ties {rows}")
    for kw in (dict(), dict(renorm=True), dict(score="sigmoid", renorm=True)):
        check_route(bnn, torch.from_numpy(l.astype(np.float32)).cuda(), top, what=str(kw), **kw)
    bias = np.zeros(E, dtype=np.float32)
    bias[4] = -np.inf                                             # an expert that is switched off
    bias[5] = np.nan
    for score in ("softmax", "sigmoid"):
        check_route(bnn, torch.from_numpy(l.astype(np.float32)).cuda(), top, score=score, bias=torch.from_numpy(bias).cuda(), what=score)


@pytest.mark.parametrize("rows,used", [(20, 0), (20, -1), (20, 7), (20, 20), (20, 99), (300, 0), (300, 1), (300, 257), (300, 300)])
def test_route_padded_batch(bnn, rows, used):
    rng = np.random.default_rng(10)
    banner(f"route used {rows} {used}")
    check_route(bnn, make(rng, (rows, 12)), 3, used=used, what=f"{rows} {used}")


def test_route_many_rows(bnn):
    """More rows than workgroups take one each, all of them to few experts."""
    rng = np.random.default_rng(11)
    l = rng.standard_normal((60000, 6)).astype(np.float32)
    l[:, 2] += 5
    banner("route 60000")
    check_route(bnn, torch.from_numpy(l).cuda(), 2, what="60000")


# ---- expert_linear


def matrices(bnn, rng, E, N, K, ternary, one_scale, bias):
    """t [E, N, K], and the same as ExpertWeights through the library's packing."""
    t = rng.integers(-1, 2, (E, N, K)) if ternary else 1 - 2 * rng.integers(0, 2, (E, N, K))
    T = torch.from_numpy(t.astype(np.float32)).cuda()
    if ternary:
        planes = [bnn.pack_weights_ternary(m, delta=0.5) for m in T]
        S, Z = torch.stack([p[0] for p in planes]), torch.stack([p[1] for p in planes])
    else:
        S, Z = torch.stack([bnn.pack_weights(m, alpha=False)[0] for m in T]), None
    alpha = 0.02 * (1 + 0.3 * make(rng, E if one_scale else (E, N)))
    b = make(rng, (E, N)) if bias else None
    return t, alpha, b, bnn.ExpertWeights(S, K, Zp=Z, alpha=alpha, bias=b)


def int8_rows(bnn, rng, rows, K):
    """Codes of all sizes; bytes past K hold anything."""
    x = torch.from_numpy(rng.integers(-128, 128, (rows, bnn.i8_ld(K))).astype(np.int8)).cuda()
    return x[:, :K]


def split(rng, P, E, how):
    """Offsets of P positions over E experts."""
    if how == "even":
        cuts = np.linspace(0, P, E + 1).astype(int)
    elif how == "one":                           # all to a single expert in the middle
        cuts = np.array([0] * (E // 2 + 1) + [P] * (E - E // 2))
    elif how == "short":                         # positions behind the last expert's
        cuts = np.sort(np.concatenate(([0], rng.integers(0, P + 1, E)))) * 3 // 4
    else:
        cuts = np.sort(np.concatenate(([0, P], rng.integers(0, P + 1, E - 1))))
        if E > 3:
            cuts[2] = cuts[1]                    # an expert without positions
    cuts[0] = 0
    return cuts.astype(np.int32)


def check_linear(bnn, rng, E, P, N, K, *, ternary=True, one_scale=True, bias=False, gated=False, act="none", out="f32", residual=False, rows=None, top=2,
                 how="ragged", xscale=True, pad=0, bad=False):
    what = f"E={E} P={P} N={N} K={K} ternary={ternary} gated={gated} act={act} out={out}"
    banner(what)
    t, alpha, b, W = matrices(bnn, rng, E, N, K, ternary, one_scale, bias)
    up = matrices(bnn, rng, E, N, K, ternary, not one_scale, bias) if gated else None
    offsets = None if E == 1 and how == "none" else split(rng, P, E, how)
    order = None
    R = P
    if rows is not None:
        R = rows
        order = rng.integers(0, R * top, P).astype(np.int32)
        if bad and P > 3:
            order[1], order[2], order[3] = -1, R * top, 2 ** 31 - 1
    Xq = int8_rows(bnn, rng, R, K)
    xs = torch.from_numpy((0.01 + 0.02 * rng.random(R)).astype(np.float32)).cuda() if xscale else None
    kind = KINDS[out]
    res = make(rng, (P, N), kind) if residual else None
    y = strided(torch.full((P, N), LEFT, dtype=kind, device="cuda"), pad)
    got = bnn.expert_linear(Xq, W, xscale=xs, offsets=None if offsets is None else torch.from_numpy(offsets).cuda(),
                            order=None if order is None else torch.from_numpy(order).cuda(), per_row=top, up=up[3] if gated else None, act=act,
                            residual=strided(res, pad), out=y)
    torch.cuda.synchronize()
    assert got is y
    want, off, live = ref.expert_linear(Xq, t, alpha, xscale=xs, bias=b, order=order, per_row=top, offsets=offsets, act=act, up=up[:3] if gated else None,
                                        residual=res)
    assert (y[torch.from_numpy(~live).cuda()] == LEFT).all(), what + ": positions without a row were written"
    near(y[torch.from_numpy(live).cuda()], want[live], off[live], kind, what)


@pytest.mark.parametrize("K", [1, 15, 16, 17, 63, 64, 65, 100, 255, 256, 257, 500, 512, 513, 1000, 1024, 2100])
@pytest.mark.parametrize("ternary", [True, False])
def test_linear_k(bnn, K, ternary):
    rng = np.random.default_rng(K)
    for P in (3, 50, 300):
        check_linear(bnn, rng, 3, P, 40, K, ternary=ternary)


@pytest.mark.parametrize("N", [1, 2, 15, 16, 17, 31, 32, 33, 64, 100, 127, 128, 129, 256, 257, 300])
@pytest.mark.parametrize("gated", [False, True])
def test_linear_n(bnn, N, gated):
    rng = np.random.default_rng(N)
    for P in (5, 70, 400):
        check_linear(bnn, rng, 2, P, N, 200, gated=gated, out="bf16" if N % 2 else "f32")


@pytest.mark.parametrize("P", [1, 2, 15, 16, 17, 31, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257, 511, 513, 1000])
@pytest.mark.parametrize("E,how", [(1, "none"), (1, "ragged"), (4, "ragged"), (5, "one"), (7, "short"), (70, "ragged"), (130, "one")])
def test_linear_positions(bnn, P, E, how):
    rng = np.random.default_rng(P)
    check_linear(bnn, rng, E, P, 48, 130, how=how, ternary=P % 2 == 0)
    check_linear(bnn, rng, E, P, 33, 96, how=how, rows=max(1, P // 2), gated=True, act="silu", ternary=P % 2 == 1)


@pytest.mark.parametrize("act", ["none", "relu", "relu2", "silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("out", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("P", [9, 300])
def test_linear_epilogues(bnn, act, out, P):
    rng = np.random.default_rng(12)
    for kw in (dict(), dict(bias=True, one_scale=False), dict(residual=True, bias=True), dict(gated=True, bias=True), dict(gated=True, residual=True, xscale=False)):
        check_linear(bnn, rng, 3, P, 72, 160, act=act, out=out, **kw)
        check_linear(bnn, rng, 3, P, 37, 160, act=act, out=out, pad=3, ternary=False, **kw)


@pytest.mark.parametrize("P", [7, 40, 500])
def test_linear_rows_of_nobody(bnn, P):
    rng = np.random.default_rng(13)
    check_linear(bnn, rng, 4, P, 50, 128, rows=6, top=3, bad=True)
    check_linear(bnn, rng, 4, P, 50, 128, rows=6, top=3, bad=True, gated=True, act="relu2")


def test_linear_large_sums(bnn):
    """K of 2^17: sums up to 2^24."""
    rng = np.random.default_rng(14)
    for P in (2, 300):
        K = 1 << 17
        T = torch.ones((1, 20, K), device="cuda")
        T[0, 3] = -1
        S, _ = bnn.pack_weights(T[0], alpha=False)
        W = bnn.ExpertWeights(S, K, alpha=torch.ones(1, device="cuda"))
        Xq = torch.full((P, K), 127, dtype=torch.int8, device="cuda")
        Xq[0] = -128
        y = bnn.expert_linear(Xq, W)
        torch.cuda.synchronize()
        want = torch.full((P, 20), 127.0 * K)
        want[0] = -128.0 * K
        want[:, 3] *= -1
        assert torch.equal(y.cpu(), want)


def test_linear_special_scales(bnn):
    """Infinities and NaN of scales and biases go where the formula takes them."""
    rng = np.random.default_rng(15)
    t, alpha, b, W = matrices(bnn, rng, 2, 20, 64, True, False, True)
    for P in (6, 300):
        Xq = int8_rows(bnn, rng, P, 64)
        Xq[2] = 0
        xs = torch.ones(P, device="cuda")
        xs[1], xs[2], xs[3] = float("inf"), float("inf"), float("nan")
        offsets = torch.tensor([0, P // 2, P], dtype=torch.int32).cuda()
        banner(f"special scales {P}")
        y = bnn.expert_linear(Xq, W, xscale=xs, offsets=offsets)
        torch.cuda.synchronize()
        y = y.cpu()
        assert torch.isnan(y[2]).all() and torch.isnan(y[3]).all() and not torch.isfinite(y[1]).any() and torch.isfinite(y[4:]).all()


@pytest.mark.parametrize("P", [4, 200])
def test_linear_residual_in_place(bnn, P):
    rng = np.random.default_rng(16)
    t, alpha, b, W = matrices(bnn, rng, 1, 64, 128, True, True, False)
    Xq, r = int8_rows(bnn, rng, P, 128), make(rng, (P, 64))
    banner(f"residual in place {P}")
    want = bnn.expert_linear(Xq, W, residual=r)
    got = bnn.expert_linear(Xq, W, residual=r, out=r)
    torch.cuda.synchronize()
    assert torch.equal(want, got)


def test_linear_agrees_with_the_layers(bnn):
    """The same numbers as bwn_i8_linear's, bit for bit."""
    rng = np.random.default_rng(17)
    for M in (1, 40, 300):
        K, N = 500, 90
        w, x = make(rng, (N, K)), make(rng, (M, K))
        g = bnn.weight_scale_tensor(w)
        S, Z, _ = bnn.pack_weights_ternary(w, gamma=g)
        q = bnn.quantize_act_i8(x)
        banner(f"against the layers {M}")
        want = bnn.bwn_i8_linear(S, K, bnn.EPI_SCALE_F32 | bnn.EPI_ALPHA_TENSOR | bnn.W_TERNARY, Zp=Z, alpha=g, **q)["Y"]
        got = bnn.expert_linear(q["Xq"], bnn.ExpertWeights(S, K, Zp=Z, alpha=g), xscale=q["xscale"])
        torch.cuda.synchronize()
        assert torch.equal(want, got)


# ---- together


class Experts:
    """A feed-forward half: norm, router, experts, and the join into the next norm."""

    def __init__(self, bnn, rng, D=192, F=320, E=6, top=2):
        self.bnn, self.top, self.E = bnn, top, E
        self.gate, self.up, self.down = (matrices(bnn, rng, E, n, k, True, True, False) for n, k in ((F, D), (F, D), (D, F)))
        self.router = make(rng, (E, D), by=0.3)
        self.w1, self.w2, self.w3 = (1 + make(rng, n, by=0.1) for n in (D, F, D))

    def __call__(self, x, attended, used):
        b = self.bnn
        n = b.block_norm(x, attended, pre_weight=self.w1, y_dtype=torch.float32, used=used)
        r = b.expert_route(n["y"] @ self.router.T, self.top, renorm=True, used=used)
        h = b.expert_linear(n["Xq"], self.gate[3], xscale=n["xscale"], offsets=r["offsets"], order=r["order"], per_row=self.top, up=self.up[3], act="silu",
                            out_dtype=torch.bfloat16)
        h = b.block_norm(branch=h, pre_weight=self.w2, used=r["offsets"][self.E:])
        d = b.expert_linear(h["Xq"], self.down[3], xscale=h["xscale"], offsets=r["offsets"])
        return n, r, h, d, b.block_norm(n["x"], d, place=r["place"], weight=r["weight"], pre_weight=self.w3, y_dtype=torch.float32, used=used)


@pytest.mark.parametrize("rows,used", [(1, 1), (9, 9), (40, 33), (600, 590)])
def test_feed_forward(bnn, rows, used):
    rng = np.random.default_rng(18)
    m = Experts(bnn, rng)
    x, att = make(rng, (rows, 192), torch.bfloat16, 2.0), make(rng, (rows, 192))
    banner(f"feed forward {rows}")
    n, r, h, d, z = m(x, att, torch.tensor([used], dtype=torch.int32).cuda())
    torch.cuda.synchronize()
    E, top, P = m.E, m.top, used * m.top
    # each step from what the step before it gave
    _, stored, v = ref.block_norm(x, att, pre_weight=m.w1)
    near(n["y"][:used], v[:used], ref.E32 * np.abs(v[:used]) + 1e-9, torch.float32, "y")
    offsets = r["offsets"].cpu().numpy()
    assert offsets[-1] == P
    order = r["order"].cpu().numpy()
    want, off, _ = ref.expert_linear(n["Xq"][:used], m.gate[0], m.gate[1], xscale=n["xscale"][:used], order=order[:P], per_row=top, offsets=offsets, act="silu", up=m.up[:3])
    hidden = torch.from_numpy(want).float().to(torch.bfloat16)
    code, scale, _ = ref.quantized(ref.norm(hidden.double().numpy(), "rms", m.w2, None, 1e-6))
    far = np.abs(h["Xq"][:P].cpu().numpy().astype(int) - code)
    assert far.max(initial=0) <= 1 and (far > 0).mean() < 0.02     # a bfloat16 of the hidden units that rounds the other way moves a code by one at most
    want, off, _ = ref.expert_linear(h["Xq"][:P], m.down[0], m.down[1], xscale=h["xscale"][:P], offsets=offsets)
    near(d[:P], want, off, torch.float32, "down")
    s, stored, v = ref.block_norm(n["x"][:used], d[:P], place=r["place"][:used], weight=r["weight"][:used], pre_weight=m.w3)
    near(z["x"][:used], s, ref.E32 * np.abs(s), torch.bfloat16, "x")


def test_another_stream(bnn):
    rng = np.random.default_rng(19)
    m = Experts(bnn, rng)
    x, att, used = make(rng, (33, 192)), make(rng, (33, 192)), torch.tensor([33], dtype=torch.int32).cuda()
    banner("another stream")
    want = m(x, att, used)[-1]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = m(x, att, used)[-1]
    side.synchronize()
    assert torch.equal(got["y"], want["y"]) and torch.equal(got["Xq"], want["Xq"])


@pytest.mark.parametrize("rows", [1, 50, 400])
def test_graph_replays(bnn, rows):
    """A captured step follows its inputs, counts included."""
    rng = np.random.default_rng(20)
    m = Experts(bnn, rng)
    x, att = make(rng, (rows, 192)), make(rng, (rows, 192))
    used = torch.tensor([rows], dtype=torch.int32).cuda()
    banner(f"graph {rows}")
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        m(x, att, used)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = m(x, att, used)[-1]
    for i in range(6):
        x.copy_(make(rng, (rows, 192)))
        att.copy_(make(rng, (rows, 192), by=1.0 + i))
        n = max(1, rows - 3 * i)
        used.fill_(n)
        want = m(x, att, used)[-1]
        want = {k: want[k][:n].clone() for k in want}
        graph.replay()
        torch.cuda.synchronize()
        for k in want:
            assert torch.equal(held[k][:n], want[k]), (i, k)


# ---- the calls again, where they are most likely to go wrong


@pytest.mark.parametrize("which", ["x", "branch"])
@pytest.mark.parametrize("factor", [0.5, -3.0, 0.3, 0.0])
@pytest.mark.parametrize("pre", ["none", "rms", "layer"])
def test_norm_factor_of_one_input(bnn, which, factor, pre):
    rng = np.random.default_rng(21)
    banner(f"norm factor {which} {factor} {pre}")
    for D in (256, 4096, 1001):
        t = make(rng, (4, D), torch.bfloat16)
        kw = dict(x_scale=factor) if which == "x" else dict(branch_scale=factor)
        check_norm(bnn, t if which == "x" else None, t if which == "branch" else None, pre=pre, what=f"{which} {factor} {pre} {D}", **kw)


def test_norm_stream_without_branch(bnn):
    """x_out where only one input is given: the stream is stored and the norm reads it as stored."""
    rng = np.random.default_rng(22)
    banner("norm x_out of one input")
    for D in (512, 777):
        for kind in (torch.bfloat16, torch.float16, torch.float32):
            x = make(rng, (5, D), kind)
            out = {"x": torch.empty_like(x), "y": torch.empty((5, D), device="cuda")}
            bnn.block_norm(x, x_scale=0.3, pre="rms", out=out)
            torch.cuda.synchronize()
            s, stored, v = ref.block_norm(x, None, x_scale=0.3)
            np.testing.assert_array_equal(ref.f64(out["x"]), stored)
            near(out["y"], v, ref.E32 * np.abs(v) + 1e-9, torch.float32, "y")
            out = {"x": torch.empty((5, D), dtype=kind, device="cuda")}
            bnn.block_norm(None, x, branch_scale=0.7, out=out)           # the branch alone, nothing but the stream asked for
            torch.cuda.synchronize()
            assert torch.equal(out["x"], (x.double() * float(np.float32(0.7))).float().to(kind))


def test_norm_rows_far_apart(bnn):
    """Rows past 2^32 bytes."""
    rng = np.random.default_rng(23)
    banner("norm rows far apart")
    M, ld, D = 40000, 1 << 16, 136
    big = torch.empty((M, ld), dtype=torch.bfloat16, device="cuda")
    x = big[:, 64: 64 + D]
    x.copy_(make(rng, (M, D), torch.bfloat16))
    got = bnn.block_norm(x, y_dtype=torch.float32)
    torch.cuda.synchronize()
    at = np.r_[0:3, M - 3: M]
    _, _, v = ref.block_norm(x[at.tolist()], None)
    near(got["y"][at.tolist()], v, ref.E32 * np.abs(v) + 1e-9, torch.float32, "y")


@pytest.mark.parametrize("K", [896, 1024, 1152, 1280, 1536, 2048, 4096, 5000])
@pytest.mark.parametrize("ternary", [True, False])
def test_linear_long_rows(bnn, K, ternary):
    """Rows of many stages: every turn of the ring and of the weight chunks."""
    rng = np.random.default_rng(K)
    for P, N in ((70, 260), (300, 40), (1100, 130)):
        check_linear(bnn, rng, 2, P, N, K, ternary=ternary, gated=N == 130, act="silu" if N == 130 else "none")


def test_linear_wide_grids(bnn):
    """128 positions to a tile: enough tiles for two workgroups to each compute unit."""
    rng = np.random.default_rng(24)
    check_linear(bnn, rng, 4, 3000, 6200, 200, ternary=True, how="even")
    check_linear(bnn, rng, 3, 4100, 4100, 140, ternary=False, gated=True, act="relu2", out="bf16", how="ragged", rows=900, top=5)


def test_linear_far_rows(bnn):
    """Rows of INT8 values past 2^31 bytes, outputs past 2^32."""
    rng = np.random.default_rng(25)
    K, R, N = 200, 20000, 48
    big = torch.zeros((R, 1 << 17), dtype=torch.int8, device="cuda")
    rows = torch.tensor([0, 5, 16383, 16384, 19998, 19999])
    big[rows.cuda(), :K] = torch.from_numpy(rng.integers(-127, 128, (6, K)).astype(np.int8)).cuda()
    t, alpha, b, W = matrices(bnn, rng, 1, N, K, True, True, False)
    for P in (6, 300):
        order = rows[torch.arange(P) % 6].to(torch.int32)
        out = torch.empty((P, 1 << 24), dtype=torch.bfloat16, device="cuda")[:, :N]
        banner(f"far rows {P}")
        bnn.expert_linear(big[:, :K], W, order=order.cuda(), out=out)
        torch.cuda.synchronize()
        want, off, _ = ref.expert_linear(big[rows.cuda()][:, :K], t, alpha, order=np.arange(P) % 6)
        near(out, want, off, torch.bfloat16, f"far rows {P}")


@pytest.mark.parametrize("P", [20, 400])
def test_linear_offsets_past_the_positions(bnn, P):
    """Offsets below 0 and past the positions count as the ends; one that decreases gives its expert no positions."""
    rng = np.random.default_rng(26)
    t, alpha, b, W = matrices(bnn, rng, 3, 40, 96, True, True, False)
    Xq = int8_rows(bnn, rng, P, 96)
    banner(f"offsets {P}")
    for raw, clean in (([-5, P // 2, P // 2, P + 100], [0, P // 2, P // 2, P]), ([0, P, P // 3, P // 3], [0, P, P, P])):
        y = torch.full((P, 40), LEFT, dtype=torch.float32, device="cuda")
        bnn.expert_linear(Xq, W, offsets=torch.tensor(raw, dtype=torch.int32).cuda(), out=y)
        torch.cuda.synchronize()
        want, off, live = ref.expert_linear(Xq, t, alpha, offsets=clean)
        near(y, want, off, torch.float32, str(raw))


def test_two_streams_at_once(bnn):
    rng = np.random.default_rng(27)
    m = Experts(bnn, rng)
    x = [make(rng, (257, 192)) for _ in range(2)]
    used = torch.tensor([257], dtype=torch.int32).cuda()
    banner("two streams")
    want = [m(a, a, used)[-1]["y"].clone() for a in x]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        got = []
        for s, a in zip(streams, x):
            with torch.cuda.stream(s):
                got.append(m(a, a, used)[-1]["y"])
        torch.cuda.synchronize()
        assert all(torch.equal(g, w) for g, w in zip(got, want))


def test_empty_calls(bnn):
    banner("empty calls")
    z = torch.empty((0, 64), device="cuda")
    assert bnn.block_norm(z, z, y_dtype=torch.bfloat16, planes=True)["y"].shape == (0, 64)
    r = bnn.expert_route(torch.empty((0, 8), device="cuda"), 2)
    torch.cuda.synchronize()
    assert r["offsets"].tolist() == [0] * 9
    W = bnn.ExpertWeights(torch.zeros((3, 4), dtype=torch.int32, device="cuda"), 100, alpha=torch.ones(1, device="cuda"))
    y = bnn.expert_linear(torch.empty((0, 112), dtype=torch.int8, device="cuda")[:, :100], W)
    assert y.shape == (0, 3)


def test_binding_checks(bnn):
    """Wrong shapes, types and devices are refused before a launch."""
    x, h = torch.zeros((4, 32), device="cuda"), torch.zeros((4, 32))
    W = bnn.ExpertWeights(torch.zeros((3, 4), dtype=torch.int32, device="cuda"), 32, alpha=torch.ones(1, device="cuda"))
    q = torch.zeros((4, 32), dtype=torch.int8, device="cuda")
    for call in (lambda: bnn.block_norm(x, h), lambda: bnn.block_norm(x, torch.zeros((4, 31), device="cuda")), lambda: bnn.block_norm(x.double()),
                 lambda: bnn.block_norm(x, pre="batch"), lambda: bnn.block_norm(x, pre_weight=torch.ones(31, device="cuda")), lambda: bnn.block_norm(x, weight=x),
                 lambda: bnn.block_norm(x.T), lambda: bnn.block_norm(x, out={"Y": x}), lambda: bnn.block_norm(x, x, place=torch.zeros((2, 2), dtype=torch.int32, device="cuda")),
                 lambda: bnn.block_norm(x, x, place=torch.zeros((4, 2), dtype=torch.int32, device="cuda"), weight=torch.ones((2, 4), device="cuda")), lambda: bnn.block_norm(x, out={"y": torch.zeros((3, 32), device="cuda")}),
                 lambda: bnn.expert_route(x, 2, score="tanh"), lambda: bnn.expert_route(x, 2, bias=torch.zeros(5, device="cuda")), lambda: bnn.expert_route(x, 33),
                 lambda: bnn.expert_linear(q, W, act="tanh"), lambda: bnn.expert_linear(q.cpu(), W), lambda: bnn.expert_linear(x, W),
                 lambda: bnn.expert_linear(q, W, xscale=torch.ones(3, device="cuda")), lambda: bnn.expert_linear(q, W, residual=torch.zeros((4, 3))),
                 lambda: bnn.expert_linear(q, W, offsets=torch.zeros(3, dtype=torch.int32, device="cuda")), lambda: bnn.expert_linear(q, W, out_dtype=torch.float64)):
        with pytest.raises((ValueError, TypeError, bnn.BnnError)):
            call()
