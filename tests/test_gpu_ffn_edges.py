"""Feed-forward calls on the GPU where they are easily wrong: far arguments of
the activations, paths that only large calls take, shared and reused memory."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import ffn_ref as ref
from gpu_util import banner
from test_gpu_ffn import KINDS, LEFT, Experts, bnn, int8_rows, make, matrices, near, split  # noqa: F401 (bnn: the fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("P", [1, 300])
@pytest.mark.parametrize("low,high", [(-115, -96), (-96, -88), (-88, -40), (-40, -20), (-20, -10), (-10, -5), (-5, 0), (0, 5), (5, 100)])
def test_silu_of_exact_arguments(bnn, P, low, high):
    """z = the bias, sums of 0.  Roundings, in half steps of fp32 (E32 of the value): exponential 2, its correction 1, product
    with z 1, sum 1, reciprocal 2, last product 1: 8.  Below the normal numbers the two products round to a
    step of their own, half of one each."""
    N = 1 << 16
    z = torch.from_numpy(np.random.default_rng(28).uniform(low, high, N).astype(np.float32)).cuda()
    W = bnn.ExpertWeights(torch.zeros((N, 4), dtype=torch.int32, device="cuda"), 16, alpha=torch.ones(1, device="cuda"), bias=z)
    banner(f"silu {P} {low} {high}")
    y = ref.f64(bnn.expert_linear(torch.zeros((P, 16), dtype=torch.int8, device="cuda"), W, act="silu"))
    want = ref.f64(z) / (1 + np.exp(-ref.f64(z)))
    off = np.abs(y - want) - 8 * ref.E32 * np.abs(want) - 2.0 ** -149
    assert off.max() <= 0, f"{(np.abs(y - want) / np.abs(want)).max() / ref.E32} half steps"


@pytest.mark.parametrize("P", [1, 300])
@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
def test_activations_at_the_ends(bnn, P, act):
    """Infinite and very large arguments: the formulas' limits; -inf times 0 is NaN in them."""
    z = torch.tensor([np.inf, 3e38, 1e30, 161.0, 0.0, -0.0, -161.0, -1e13, -1e30, -3e38, -np.inf, np.nan], device="cuda")
    W = bnn.ExpertWeights(torch.zeros((12, 4), dtype=torch.int32, device="cuda"), 16, alpha=torch.ones(1, device="cuda"), bias=z)
    banner(f"ends {P} {act}")
    y = bnn.expert_linear(torch.zeros((P, 16), dtype=torch.int8, device="cuda"), W, act=act)[P - 1].cpu()
    assert torch.equal(y[:4], z[:4].cpu()) and (y[4:10] == 0).all() and torch.isnan(y[10:]).all()


def tiles_of_128(E, P, N, gated):
    """Whether the products take tiles of 128 positions: 96 rows to an expert, and two workgroups to each compute unit."""
    cols = 128 if gated else 256
    return P // E >= 96 and (P + min(E, P) * 127) // 128 * -(-N // cols) >= 512


@pytest.mark.parametrize("E,P,N,K", [(4, 3000, 6200, 768), (4, 3000, 6200, 896), (4, 3000, 6200, 1024), (4, 3000, 6200, 1152), (4, 3000, 6200, 1300), (2, 3000, 6200, 1408),
                                     (2, 3000, 6200, 2100), (2, 3000, 6200, 4096)])
@pytest.mark.parametrize("ternary", [True, False])
@pytest.mark.parametrize("gated", [False, True])
def test_linear_long_rows_of_wide_grids(bnn, E, P, N, K, ternary, gated):
    """Tiles of 128 positions over many stages, one turn of the ring and several, whole and with a rest: every output.
    The sums are whole numbers, and products, comparisons and the last rounding are the same in torch, bit for bit."""
    rng = np.random.default_rng(K)
    if gated:
        N //= 2
    assert tiles_of_128(E, P, N, gated)
    banner(f"wide grid E={E} P={P} N={N} K={K} ternary={ternary} gated={gated}")
    mats = [matrices(bnn, rng, E, N, K, ternary, h == 0, h == 1) for h in range(2 if gated else 1)]
    R, top = (700, 5) if gated else (P, 1)
    order = torch.from_numpy(rng.integers(0, R * top, P).astype(np.int32)).cuda() if gated else None
    offsets = split(rng, P, E, "ragged")
    Xq = int8_rows(bnn, rng, R, K)
    xs = torch.from_numpy((0.01 + 0.02 * rng.random(R)).astype(np.float32)).cuda()
    kind = torch.bfloat16 if gated else torch.float32
    got = bnn.expert_linear(Xq, mats[0][3], xscale=xs, offsets=torch.from_numpy(offsets).cuda(), order=order, per_row=top, up=mats[1][3] if gated else None,
                            act="relu2" if gated else "none", out_dtype=kind)
    torch.cuda.synchronize()
    row = (order // top).long() if gated else torch.arange(P, device="cuda")
    for e in range(E):
        at = row[offsets[e]:offsets[e + 1]]
        x, z = Xq[at].double(), []
        for t, alpha, bias, _ in mats:
            D = torch.matmul(x, torch.from_numpy(t[e]).cuda().double().t().contiguous()).float()
            v = alpha[e] * D * xs[at][:, None]
            z.append(v if bias is None else v + bias[e])
        want = z[0]
        if gated:
            want = torch.where(want < 0, torch.zeros_like(want), want * want) * z[1]
        assert torch.equal(got[offsets[e]:offsets[e + 1]], want.to(kind)), f"expert {e}"


@pytest.mark.parametrize("E", [2, 5])
@pytest.mark.parametrize("P", [6, 300])
def test_linear_shared_scales(bnn, E, P):
    """One row of scales for all experts, expanded; more experts than columns too."""
    rng = np.random.default_rng(29)
    for N in (40, 3):
        t, _, _, W = matrices(bnn, rng, E, N, 96, True, False, False)
        row = 0.02 * (1 + 0.3 * make(rng, N))
        planes = [bnn.pack_weights_ternary(m, delta=0.5) for m in torch.from_numpy(t.astype(np.float32)).cuda()]
        W = bnn.ExpertWeights(torch.stack([p[0] for p in planes]), 96, Zp=torch.stack([p[1] for p in planes]), alpha=row.expand(E, N))
        Xq, offsets = int8_rows(bnn, rng, P, 96), split(rng, P, E, "ragged")
        banner(f"shared scales E={E} P={P} N={N}")
        y = bnn.expert_linear(Xq, W, offsets=torch.from_numpy(offsets).cuda())
        torch.cuda.synchronize()
        want, off, _ = ref.expert_linear(Xq, t, row.expand(E, N).contiguous(), offsets=offsets)
        near(y, want, off, torch.float32, f"shared scales {N}")


def test_route_workspace_used_again(bnn):
    """One workspace, larger than most calls need, with what the last call left in it."""
    rng = np.random.default_rng(30)
    work = bnn.expert_route_workspace(5000, 200, 8)
    work.fill_(255)
    for rows, E, top in ((5000, 200, 8), (40, 7, 2), (33, 200, 5), (5000, 3, 1), (1, 200, 8), (700, 64, 6), (4100, 130, 8)):
        l = make(rng, (rows, E))
        banner(f"workspace again {rows} {E}")
        got = bnn.expert_route(l, top, workspace=work)
        torch.cuda.synchronize()
        expert, weight, offsets, order, place = ref.expert_route(l, top)
        for name, want in (("expert", expert), ("offsets", offsets), ("order", order), ("place", place)):
            np.testing.assert_array_equal(got[name].cpu().numpy(), want, err_msg=f"{name} {rows} {E}")
    for bad in (work.cpu(), work[::2], torch.empty(0, dtype=torch.uint8)):
        with pytest.raises(ValueError, match="workspace"):
            bnn.expert_route(make(rng, (100, 8)), 2, workspace=bad)
    with pytest.raises(bnn.BnnError):
        bnn.expert_route(make(rng, (100, 8)), 2, workspace=work[:16])


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("pre", ["none", "rms", "layer"])
@pytest.mark.parametrize("D", [96, 1001, 4096])
def test_norm_scale_is_of_the_rows_before_they_are_rounded(bnn, kind, pre, D):
    """xscale with a 16-bit y: max |v| of the 64-bit rows / 127, fp32 roundings of v and of the quotient."""
    rng = np.random.default_rng(31)
    x, b = make(rng, (6, D), by=3.0), make(rng, (6, D), KINDS[kind])
    banner(f"xscale {kind} {pre} {D}")
    got = bnn.block_norm(x, b, pre=pre, y_dtype=KINDS[kind])
    torch.cuda.synchronize()
    _, stored, v = ref.block_norm(x, b, pre=pre)
    most = np.abs(v).max(-1)
    assert (np.abs(ref.f64(got["xscale"]) - most / 127) <= 2.01 * ref.E32 * most / 127).all()
    near(got["y"], v, ref.E32 * np.abs(v) + 2.0 ** -40 * most[:, None], KINDS[kind], "y")


@pytest.mark.parametrize("rows,used", [(1, 1), (9, 9), (40, 33), (600, 590)])
def test_feed_forward_into_the_next_block(bnn, rows, used):
    """The join at the end of a step: its norm and its INT8 rows, from what the products gave."""
    rng = np.random.default_rng(18)
    m = Experts(bnn, rng)
    x, att = make(rng, (rows, 192), torch.bfloat16, 2.0), make(rng, (rows, 192))
    banner(f"next block {rows}")
    n, r, h, d, z = m(x, att, torch.tensor([used], dtype=torch.int32).cuda())
    torch.cuda.synchronize()
    s, _, _ = ref.block_norm(n["x"][:used], d[:used * m.top], place=r["place"][:used], weight=r["weight"][:used], pre_weight=m.w3)
    near(z["x"][:used], s, ref.E32 * np.abs(s), torch.bfloat16, "x")
    v = ref.norm(ref.f64(z["x"][:used]), "rms", m.w3, None, 1e-6)      # the norm reads the stream as it is stored
    near(z["y"][:used], v, ref.E32 * np.abs(v) + 2.0 ** -40 * np.abs(v).max(-1, keepdims=True), torch.float32, "y")
    code, scale, _ = ref.quantized(z["y"][:used].cpu().numpy())
    np.testing.assert_array_equal(z["Xq"][:used].cpu().numpy(), code)
    np.testing.assert_array_equal(z["xscale"][:used].cpu().numpy(), scale)


@pytest.mark.parametrize("rows", [20, 300])
@pytest.mark.parametrize("renorm", [False, True])
def test_route_small_scores(bnn, rows, renorm):
    """Sigmoids of logits from -87 to -103: numbers below the normal ones, not zeros.  Roundings, in half steps of fp32:
    exponential 2, sum 1, quotient 1, and a step or two of the smallest number, d; the renormalized ones from scores w, w_i off by
    that much each: a quotient of w + d and their sum."""
    rng = np.random.default_rng(32)
    l = torch.from_numpy(rng.uniform(-103, -87, (rows, 40)).astype(np.float32)).cuda()
    l[3] = -200.0                                                # nothing left: weights 0
    banner(f"small scores {rows} {renorm}")
    got = bnn.expert_route(l, 4, score="sigmoid", renorm=renorm)
    torch.cuda.synchronize()
    w = np.exp(-np.sort(-ref.f64(l), 1)[:, :4])
    d = 4 * ref.E32 * w + 2 * 2.0 ** -149
    have = ref.f64(got["weight"])
    if renorm:
        live = w.sum(1) > 2.0 ** -140
        assert live.sum() > rows / 2
        total = w.sum(1, keepdims=True)
        assert (np.abs(have - w / total) <= (d + w / total * d.sum(1, keepdims=True)) / (total - d.sum(1, keepdims=True)) + 6 * ref.E32)[live].all()
        assert (np.abs(have[live].sum(1) - 1) <= 16 * ref.E32).all()
    else:
        assert (np.abs(have - w) <= d).all()
    assert (have[3] == 0).all()


@pytest.mark.parametrize("M,D", [((1 << 23) + 3, 2), ((1 << 20) + 5, 516)])
def test_norm_more_workgroups_than_one_dimension(bnn, M, D):
    """Past 2^20 workgroups a launch has two dimensions: four rows to each, and one."""
    banner(f"norm {M} x {D}")
    x = (torch.arange(M * D, device="cuda", dtype=torch.int32) % 251 - 125).reshape(M, D).to(torch.bfloat16)
    used = torch.tensor([M - 2], dtype=torch.int32).cuda()
    out = {"y": torch.full((M, D), LEFT, dtype=torch.bfloat16, device="cuda")}
    bnn.block_norm(x, x_scale=0.5, pre="none", used=used, out=out)
    torch.cuda.synchronize()
    assert torch.equal(out["y"][:M - 2], x[:M - 2] * 0.5) and (out["y"][M - 2:] == LEFT).all()


def test_linear_more_workgroups_than_one_dimension(bnn):
    """2^24 outputs of few rows: 2^21 workgroups.  K = 1, so that y is a product of numbers."""
    N, P = 1 << 24, 80
    banner("linear 2^21 workgroups")
    gen = torch.Generator(device="cuda").manual_seed(33)
    q = torch.zeros((P, 16), dtype=torch.int8, device="cuda")
    q[:, 0] = torch.arange(P, device="cuda") - 40
    offsets = torch.tensor([0, 47, P], dtype=torch.int32, device="cuda")
    weights, signs = [], []
    for _ in range(2):
        S, Z = (torch.randint(0, 2, (2, N, 4), dtype=torch.int32, device="cuda", generator=gen) for _ in range(2))
        alpha = torch.tensor([0.5, 2.0], device="cuda")
        weights.append(bnn.ExpertWeights(S, 1, Zp=Z, alpha=alpha))
        signs.append((Z[:, :, 0] * (1 - 2 * S[:, :, 0])).to(torch.int8))
        del S, Z
    y = bnn.expert_linear(q[:, :1], weights[0], offsets=offsets, up=weights[1], out_dtype=torch.bfloat16)
    torch.cuda.synchronize()
    for p in range(P):
        e = int(p >= 47)
        d = (signs[0][e] * signs[1][e]).to(torch.bfloat16) * float((p - 40) ** 2 * (0.25, 4.0)[e])     # a product of fp32 numbers, rounded once
        assert torch.equal(y[p], d), p
