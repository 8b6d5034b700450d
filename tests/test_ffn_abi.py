"""Feed-forward calls without a GPU: every refusal of the C ABI comes before a
launch; sizes of the laid-out weights and of the workspace; the definitions in
64 bits against plain torch."""
from __future__ import annotations

import ctypes
import math

import numpy as np
import pytest
import torch

import ffn_ref as ref

OK, ERR_NULL, ERR_SHAPE, ERR_LD, ERR_ALIGN, ERR_UNSUPPORTED = range(6)
A16, A8, A4, A2, A1 = 0x10000, 0x10008, 0x10004, 0x10002, 0x10001    # fake device addresses: nothing below is launched
F32, BF16, F16 = 3, 1, 2
BIG = 1 << 62


@pytest.fixture(scope="module")
def bnn():
    import xnor_popcount_gemm_amd as m
    m.lib()
    return m


NORM = dict(M=0, D=100, used=A16, x=A16, ldx=100, x_dtype=BF16, branch=A16, ldb=104, b_dtype=F32, b_rows=7, place=A16, weight=A16, parts=2, post=1,
            post_weight=A16, post_bias=A16, gate=A16, ld_gate=0, x_scale=1.0, branch_scale=1.0, pre=2, pre_weight=A16, pre_bias=A16, eps=1e-6,
            x_out=A16, ldxo=100, y=A16, ldy=100, y_dtype=F16, Xq=A16, ldXq=112, Xb=A16, ldXb=4, xsum=A16, xscale=A16)
ROUTE = dict(logits=A16, ld=8, dtype=F32, rows=100, experts=8, top=2, used=A16, score=0, bias=A16, renorm=1, scale=1.0, expert=A16, weight=A16,
             offsets=A16, order=A16, place=A16, workspace=A16, workspace_bytes=1 << 30)
LINEAR = dict(Xq=A16, ldXq=128, xscale=A16, rows=5, order=A16, per_row=2, offsets=A16, experts=4, positions=0, N=30, K=100, ternary=1, act=3,
              residual=A16, ldr=30, y=A16, ldy=30, y_dtype=F32)
MATRIX = dict(W=A16, alpha=A16, ld_alpha=30, bias=A16, ld_bias=30)


def fill(struct, base, kw):
    s = struct()
    for k, v in {**base, **kw}.items():
        setattr(s, k, v)
    return s


def norm(bnn, **kw):
    a = fill(bnn._NormArgs, NORM, kw)
    return bnn.lib().bnn_block_norm(ctypes.addressof(a), None)


def route(bnn, **kw):
    a = fill(bnn._RouteArgs, ROUTE, kw)
    return bnn.lib().bnn_expert_route(ctypes.addressof(a), None)


def linear(bnn, main={}, up={}, **kw):
    a = fill(bnn._ExpertArgs, LINEAR, kw)
    a.main, a.up = fill(bnn._ExpertMatrix, MATRIX, main), fill(bnn._ExpertMatrix, MATRIX, up)
    return bnn.lib().bnn_expert_linear(ctypes.addressof(a), None)


@pytest.mark.parametrize("kw,want", [
    (dict(), OK), (dict(M=-1), ERR_SHAPE), (dict(M=(1 << 30) + 1), ERR_SHAPE), (dict(D=0), ERR_SHAPE), (dict(D=16385, ldx=1 << 15), ERR_SHAPE),
    (dict(x=0, branch=0), ERR_NULL), (dict(x=0), OK), (dict(x_dtype=0), ERR_UNSUPPORTED), (dict(x_dtype=4), ERR_UNSUPPORTED), (dict(b_dtype=7), ERR_UNSUPPORTED),
    (dict(y_dtype=0), ERR_UNSUPPORTED), (dict(x=0, x_out=0, x_dtype=0), OK), (dict(x=0, x_dtype=0), ERR_UNSUPPORTED), (dict(y=0, y_dtype=0), OK),
    (dict(post=3), ERR_UNSUPPORTED), (dict(pre=-1), ERR_UNSUPPORTED), (dict(x_scale=math.inf), ERR_UNSUPPORTED), (dict(branch_scale=math.nan), ERR_UNSUPPORTED),
    (dict(eps=-1e-6), ERR_UNSUPPORTED), (dict(eps=math.nan), ERR_UNSUPPORTED), (dict(eps=math.inf), ERR_UNSUPPORTED),
    (dict(branch=0), ERR_UNSUPPORTED), (dict(branch=0, place=0), ERR_UNSUPPORTED), (dict(branch=0, place=0, gate=0), ERR_UNSUPPORTED),
    (dict(branch=0, place=0, gate=0, post=0), OK),
    (dict(x_out=0, y=0, Xq=0, Xb=0, xsum=0, xscale=0), ERR_NULL), (dict(xscale=0), ERR_NULL), (dict(xsum=0), ERR_NULL), (dict(Xb=0, xsum=0), OK),
    (dict(Xq=0, Xb=0), ERR_NULL), (dict(Xq=0, Xb=0, xsum=0, xscale=0), OK),
    (dict(ldx=99), ERR_LD), (dict(ldb=99), ERR_LD), (dict(ldxo=99), ERR_LD), (dict(ldy=99), ERR_LD), (dict(ldXq=99), ERR_LD), (dict(ldXb=3), ERR_LD),
    (dict(ldXb=6), ERR_ALIGN), (dict(ldx=BIG), ERR_LD), (dict(ld_gate=50), ERR_LD), (dict(ld_gate=100), OK),
    (dict(x=A1), ERR_ALIGN), (dict(x=A2), OK), (dict(branch=A2), ERR_ALIGN), (dict(branch=A4), OK), (dict(y=A1), ERR_ALIGN), (dict(x_out=A1), ERR_ALIGN),
    (dict(Xb=A8), ERR_ALIGN), (dict(Xq=A1), OK), (dict(gate=A2), ERR_ALIGN), (dict(gate=A4), OK), (dict(used=A2), ERR_ALIGN), (dict(place=A2), ERR_ALIGN),
    (dict(weight=A2), ERR_ALIGN), (dict(post_weight=A2), ERR_ALIGN), (dict(post_bias=A2), ERR_ALIGN), (dict(pre_weight=A2), ERR_ALIGN),
    (dict(pre_bias=A2), ERR_ALIGN), (dict(xsum=A2), ERR_ALIGN), (dict(xscale=A2), ERR_ALIGN),
    (dict(parts=0), ERR_SHAPE), (dict(parts=65), ERR_SHAPE), (dict(place=0, parts=0), OK), (dict(b_rows=-1), ERR_SHAPE), (dict(b_rows=0), OK),
    (dict(place=0, M=8), ERR_SHAPE),
])
def test_norm_refusals(bnn, kw, want):
    assert norm(bnn, **kw) == want
    assert bnn.lib().bnn_block_norm(None, None) == ERR_NULL


@pytest.mark.parametrize("kw,want", [
    (dict(rows=-1), ERR_SHAPE), (dict(rows=1 << 30), ERR_SHAPE), (dict(experts=0), ERR_SHAPE), (dict(experts=1025, ld=2000), ERR_SHAPE), (dict(top=0), ERR_SHAPE),
    (dict(top=9), ERR_SHAPE), (dict(experts=100, ld=100, top=65), ERR_SHAPE), (dict(dtype=0), ERR_UNSUPPORTED), (dict(score=2), ERR_UNSUPPORTED),
    (dict(scale=math.nan), ERR_UNSUPPORTED), (dict(ld=7), ERR_LD), (dict(ld=BIG), ERR_LD), (dict(logits=0), ERR_NULL), (dict(logits=A2), ERR_ALIGN),
    (dict(expert=0), ERR_NULL), (dict(weight=0), ERR_NULL), (dict(offsets=0), ERR_NULL), (dict(order=0), ERR_NULL), (dict(place=0), ERR_NULL),
    (dict(expert=A2), ERR_ALIGN), (dict(weight=A2), ERR_ALIGN), (dict(offsets=A2), ERR_ALIGN), (dict(order=A2), ERR_ALIGN), (dict(place=A2), ERR_ALIGN),
    (dict(used=A2), ERR_ALIGN), (dict(bias=A2), ERR_ALIGN), (dict(workspace=0), ERR_NULL), (dict(workspace=A8), ERR_ALIGN), (dict(workspace_bytes=1), ERR_SHAPE),
])
def test_route_refusals(bnn, kw, want):
    assert route(bnn, **kw) == want
    assert bnn.lib().bnn_expert_route(None, None) == ERR_NULL


@pytest.mark.parametrize("kw,want", [
    (dict(), OK), (dict(experts=0), ERR_SHAPE), (dict(experts=1025), ERR_SHAPE), (dict(positions=-1), ERR_SHAPE), (dict(positions=(1 << 30) + 1), ERR_SHAPE),
    (dict(rows=-1), ERR_SHAPE), (dict(N=-1), ERR_SHAPE), (dict(N=(1 << 24) + 1), ERR_SHAPE), (dict(K=0), ERR_SHAPE), (dict(K=(1 << 17) + 1), ERR_SHAPE),
    (dict(offsets=0), ERR_NULL), (dict(offsets=0, experts=1), OK), (dict(act=-1), ERR_UNSUPPORTED), (dict(act=6), ERR_UNSUPPORTED), (dict(y_dtype=0), ERR_UNSUPPORTED),
    (dict(per_row=0), ERR_SHAPE), (dict(order=0, per_row=0), OK), (dict(order=0, positions=6), ERR_SHAPE), (dict(Xq=0), ERR_NULL), (dict(Xq=A8), ERR_ALIGN),
    (dict(ldXq=96), ERR_LD), (dict(ldXq=120), ERR_ALIGN), (dict(xscale=A2), ERR_ALIGN), (dict(order=A2), ERR_ALIGN), (dict(offsets=A2), ERR_ALIGN),
    (dict(residual=A2), ERR_ALIGN), (dict(ldr=29), ERR_LD), (dict(residual=0, ldr=0), OK), (dict(y=0), ERR_NULL), (dict(y=A2), ERR_ALIGN),
    (dict(y=A2, residual=A2, y_dtype=BF16), OK), (dict(ldy=29), ERR_LD), (dict(ldy=BIG), ERR_LD),
    (dict(main=dict(W=0)), ERR_NULL), (dict(main=dict(W=A8)), ERR_ALIGN), (dict(main=dict(alpha=0)), ERR_NULL), (dict(main=dict(alpha=A2)), ERR_ALIGN),
    (dict(main=dict(ld_alpha=29)), ERR_LD), (dict(main=dict(ld_alpha=0)), OK), (dict(main=dict(bias=A2)), ERR_ALIGN), (dict(main=dict(ld_bias=29)), ERR_LD),
    (dict(main=dict(bias=0, ld_bias=0)), OK), (dict(up=dict(W=0, alpha=0)), OK), (dict(up=dict(alpha=0)), ERR_NULL), (dict(up=dict(W=A4)), ERR_ALIGN),
    (dict(up=dict(bias=A1)), ERR_ALIGN), (dict(positions=1 << 30, N=1 << 24, ldr=1 << 24, ldy=1 << 24, main=dict(ld_alpha=0, ld_bias=1 << 24), up=dict(W=0)), ERR_SHAPE),
])
def test_linear_refusals(bnn, kw, want):
    assert linear(bnn, **kw) == want
    assert bnn.lib().bnn_expert_linear(None, None) == ERR_NULL


def test_pack_refusals(bnn):
    def pack(Wp=A16, Zp=A16, ld=4, apart=400, E=2, N=0, K=100, out=A16, have=1 << 40):
        return bnn.lib().bnn_expert_pack(Wp, Zp, ld, apart, E, N, K, out, have, None)

    assert pack() == OK and pack(E=0) == OK and pack(Zp=0) == OK
    assert pack(E=-1) == pack(E=1025) == pack(N=-1) == pack(K=0) == pack(K=(1 << 17) + 1) == ERR_SHAPE
    assert pack(Wp=0) == pack(out=0) == ERR_NULL
    assert pack(ld=3) == pack(N=101) == pack(apart=-1) == pack(ld=BIG) == ERR_LD
    assert pack(Wp=A8) == pack(Zp=A8) == pack(out=A8) == pack(ld=6) == ERR_ALIGN
    assert pack(N=100, have=7 * 1024 * 2 - 1) == ERR_SHAPE


@pytest.mark.parametrize("E,N,K,ternary,want", [(1, 16, 256, 1, 1024), (1, 16, 512, 0, 1024), (3, 17, 257, 1, 3 * 2 * 2 * 1024), (0, 5, 5, 0, 0), (1, 1, 1, 0, 1024),
                                                (8, 4096, 4096, 1, 8 * 4096 * 4096 // 4), (8, 4096, 4096, 0, 8 * 4096 * 4096 // 8), (1, 1, 0, 0, -1), (1025, 1, 1, 0, -1)])
def test_pack_bytes(bnn, E, N, K, ternary, want):
    assert bnn.lib().bnn_expert_pack_bytes(E, N, K, ternary) == want


def test_route_workspace(bnn):
    f = bnn.lib().bnn_expert_route_workspace
    assert f(-1, 8, 2) == f(10, 0, 1) == f(10, 8, 9) == f(10, 1025, 1) == f(1 << 29, 8, 2) == -1
    last = 0
    for rows in (0, 1, 64, 65, 1000, 20000, 1 << 20):
        assert f(rows, 128, 8) >= last
        last = f(rows, 128, 8)
    assert f(1, 8, 2) == 0 and last <= 256 * 128 * 4


def test_binding_refuses_host_tensors(bnn):
    x = torch.zeros(4, 8)
    with pytest.raises(ValueError):
        bnn.block_norm(x)
    with pytest.raises(ValueError):
        bnn.block_norm()
    with pytest.raises(ValueError):
        bnn.expert_route(x, 2)
    with pytest.raises(ValueError):
        bnn.ExpertWeights(torch.zeros((4, 4), dtype=torch.int32), 100, alpha=torch.zeros(4))
    with pytest.raises(ValueError):
        bnn.expert_route_workspace(10, 8, 9)


def test_layouts(bnn):
    for struct, last in ((bnn._NormArgs, "xscale"), (bnn._RouteArgs, "workspace_bytes"), (bnn._ExpertArgs, "y_dtype")):
        assert struct._fields_[-1][0] == last
    assert ctypes.sizeof(bnn._ExpertMatrix) == 40


# ---- the definitions


def test_reference_norms():
    g = torch.Generator().manual_seed(0)
    x, b, w, c = (torch.randn(s, generator=g) for s in ((5, 40), (5, 40), (40,), (40,)))
    s, stored, y = ref.block_norm(x, b, post="rms", post_weight=w, gate=c, pre="layer", pre_weight=w, pre_bias=c, eps=1e-5, x_scale=0.5, branch_scale=2.0)
    post = torch.nn.functional.rms_norm(b.double(), (40,), w.double(), 1e-5)
    want = 0.5 * x.double() + 2 * c.double() * post
    np.testing.assert_allclose(s, want.numpy(), rtol=1e-6, atol=1e-7)      # eps is an fp32 number in one of them
    want = torch.nn.functional.layer_norm(torch.from_numpy(stored), (40,), w.double(), c.double(), 1e-5)
    np.testing.assert_allclose(y, want.numpy(), rtol=1e-6, atol=1e-7)
    place = torch.tensor([[0, 4], [-1, 2], [9, -5]])
    s, _, _ = ref.block_norm(None, b, place=place, weight=torch.ones(3, 2))
    np.testing.assert_allclose(s, torch.stack((b[0].double() + b[4], b[2].double(), 0 * b[0].double())).numpy())


def test_reference_quantizer():
    import oracle
    x = np.random.default_rng(0).standard_normal((6, 77)).astype(np.float32)
    x[2], x[3, 4], x[4, 5] = 0, np.nan, np.inf
    q, s = oracle.quantize_absmax_i8(x)
    mine = ref.quantized(x, by_quotient=True)
    np.testing.assert_array_equal(q, mine[0])
    np.testing.assert_array_equal(s, mine[1])
    planes, total = oracle.pack_planes_i8(q)[:2]
    np.testing.assert_array_equal(planes.view(np.int32), ref.planes(q, planes.shape[2]))


def test_reference_route():
    l = torch.randn((50, 12), generator=torch.Generator().manual_seed(1))
    expert, weight, offsets, order, place = ref.expert_route(l, 3, renorm=True)
    p = torch.softmax(l.double(), -1).topk(3, -1)
    np.testing.assert_array_equal(expert, p.indices.numpy())
    np.testing.assert_allclose(weight, (p.values / p.values.sum(-1, keepdim=True)).numpy())
    flat = torch.from_numpy(expert).flatten()
    np.testing.assert_array_equal(order, flat.sort(stable=True).indices.numpy())
    np.testing.assert_array_equal(offsets[1:], torch.bincount(flat, minlength=12).cumsum(0).numpy())
    np.testing.assert_array_equal(place.reshape(-1)[order], np.arange(150))
    expert, weight, offsets, order, place = ref.expert_route(torch.tensor([[-math.inf, 1.0, math.nan], [2.0, 2.0, 2.0]]), 2, used=1)
    assert expert.tolist() == [[1, -1], [-9, -9]] and place.tolist() == [[0, -1], [-9, -9]] and offsets.tolist() == [0, 0, 1, 1] and order.tolist() == [0]


def test_reference_linear():
    g = np.random.default_rng(2)
    q = torch.from_numpy(g.integers(-128, 128, (6, 30)).astype(np.int8))
    t = g.integers(-1, 2, (2, 9, 30))
    a = torch.rand((2, 9), generator=torch.Generator().manual_seed(3))
    y, off, live = ref.expert_linear(q, t, a, order=np.array([0, 11, 5, 3, 40]), per_row=2, offsets=[0, 2, 5], act="gelu", up=(t, a, None))
    rows, e = [0, 5, 2, 1], [0, 0, 1, 1]
    z = np.stack([(q[r].double().numpy() @ t[i].T) * a[i].double().numpy() for r, i in zip(rows, e)])
    want = torch.nn.functional.gelu(torch.from_numpy(z)).numpy() * z
    np.testing.assert_allclose(y[:4], want, rtol=1e-12, atol=1e-12)
    assert live.tolist() == [True] * 4 + [False]
    for act, f in (("silu", torch.nn.functional.silu), ("gelu_tanh", lambda v: torch.nn.functional.gelu(v, approximate="tanh")), ("relu2", lambda v: torch.relu(v) ** 2)):
        x = np.linspace(-9, 9, 181)
        np.testing.assert_allclose(ref.activated(x, act), f(torch.from_numpy(x)).numpy(), rtol=1e-9, atol=1e-13)
