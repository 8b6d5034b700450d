"""Cache calls without a GPU: every refusal of the C ABI comes before a launch,
the binding's own checks, and the two host functions (rotation table, tree
masks) against their definitions."""
from __future__ import annotations

import ctypes
import math

import numpy as np
import pytest
import torch

import cache_ref as ref

OK, ERR_NULL, ERR_SHAPE, ERR_LD, ERR_ALIGN, ERR_UNSUPPORTED = range(6)
A16, A8, A4, A2 = 0x10000, 0x10008, 0x10004, 0x10002    # fake device addresses: nothing below is launched


@pytest.fixture(scope="module")
def bnn():
    import xnor_popcount_gemm_amd as m
    m.lib()
    return m


def fill(struct, base, kw):
    s = struct()
    for k, v in {**base, **kw}.items():
        setattr(s, k, v)
    return s


CACHE = dict(K=A16, k_page=16 * 2 * 64, k_slot=2 * 64, k_head=64, V=A16, v_page=16 * 2 * 64, v_slot=2 * 64, v_head=64, table=A16, ld_table=4,
             num_pages=9, page_size=16, kv_heads=2, dim=64, dtype=1)
BATCH = dict(indptr=A16, ctx=A16, B=2, rows=5, max_nodes=4, max_ctx=50)
ROPE = dict(q=A16, q_row=256, q_head=64, k=A16, k_row=128, k_head=64, v=A16, v_row=128, v_head=64, src_dtype=3, heads=4, q_out=A16, qo_row=256,
            qo_head=64, positions=A16, turns=A16, max_pos=100, rot=64, interleaved=0, q_weight=A16, k_weight=A16, eps=1e-6, pos=A16, score=A16,
            ld_slots=64)
ATTN = dict(q=A16, q_row=256, q_head=64, heads=4, mask=A16, ld_mask=1, scale=0.1, out=A16, o_row=256, o_head=64, out_dtype=3, lse=A16, ld_lse=4,
            workspace=A16, workspace_bytes=1 << 40)
SCORE = dict(q=A16, q_row=256, q_head=64, heads=4, lse=A16, ld_lse=4, mask=A16, ld_mask=1, accept=A16, ld_accept=1, scale=0.1, score_in=A16,
             score_out=A16, ld_slots=64)
EVICT = dict(accept=A16, ld_accept=1, budget=32, recent=4, pos_in=A16, pos_out=A16, score_in=A16, score_out=A16, ld_slots=64, ctx_out=A16,
             workspace=A16, workspace_bytes=1 << 40)
CALLS = {"rope": ("bnn_qk_norm_rope", "_RopeArgs", ROPE), "attn": ("bnn_tree_attention", "_AttnArgs", ATTN),
         "score": ("bnn_cache_score_add", "_ScoreArgs", SCORE), "evict": ("bnn_cache_evict", "_EvictArgs", EVICT)}


def call(bnn, op, cache={}, batch={}, **kw):
    name, struct, base = CALLS[op]
    c, b, a = fill(bnn._KvCache, CACHE, cache), fill(bnn._KvBatch, BATCH, batch), fill(getattr(bnn, struct), base, kw)
    return getattr(bnn.lib(), name)(ctypes.addressof(c), ctypes.addressof(b), ctypes.addressof(a), None)


NONE = dict(B=0)   # an empty call: validated like any other, nothing launched


@pytest.mark.parametrize("op", CALLS)
def test_empty_calls_and_null_structs(bnn, op):
    assert call(bnn, op, batch=NONE) == OK
    name, struct, base = CALLS[op]
    c, b, a = fill(bnn._KvCache, CACHE, {}), fill(bnn._KvBatch, BATCH, NONE), fill(getattr(bnn, struct), base, {})
    p = [ctypes.addressof(x) for x in (c, b, a)]
    for i in range(3):
        assert getattr(bnn.lib(), name)(*[None if j == i else x for j, x in enumerate(p)], None) == ERR_NULL


@pytest.mark.parametrize("op", CALLS)
@pytest.mark.parametrize("kw,want", [
    (dict(K=0), ERR_NULL), (dict(V=0), ERR_NULL), (dict(K=A8), ERR_ALIGN), (dict(V=A4), ERR_ALIGN), (dict(table=A2), ERR_ALIGN),
    (dict(dtype=3), ERR_UNSUPPORTED), (dict(dtype=0), ERR_UNSUPPORTED), (dict(dim=80), ERR_UNSUPPORTED), (dict(dim=0), ERR_UNSUPPORTED),
    (dict(page_size=0), ERR_SHAPE), (dict(num_pages=-1), ERR_SHAPE), (dict(num_pages=1 << 31), ERR_SHAPE), (dict(kv_heads=0), ERR_SHAPE),
    (dict(ld_table=0), ERR_LD), (dict(page_size=1 << 20, ld_table=1 << 20), ERR_SHAPE), (dict(page_size=1 << 31), ERR_SHAPE),
    (dict(k_head=-64), ERR_LD), (dict(v_slot=1 << 50), ERR_LD), (dict(k_page=1 << 46, num_pages=1 << 20), ERR_LD), (dict(k_slot=132), ERR_ALIGN),
    (dict(v_head=68), ERR_ALIGN),
])
def test_cache_refusals(bnn, op, kw, want):
    assert call(bnn, op, cache=kw, batch=NONE) == want


@pytest.mark.parametrize("op", CALLS)
@pytest.mark.parametrize("kw,want", [
    (dict(indptr=0), ERR_NULL), (dict(ctx=0), ERR_NULL), (dict(indptr=A2), ERR_ALIGN), (dict(ctx=A2), ERR_ALIGN), (dict(B=-1), ERR_SHAPE),
    (dict(B=65536), ERR_SHAPE), (dict(rows=-1), ERR_SHAPE), (dict(max_nodes=-1), ERR_SHAPE), (dict(max_ctx=-1), ERR_SHAPE),
    (dict(max_ctx=1 << 31), ERR_SHAPE),
])
def test_batch_refusals(bnn, op, kw, want):
    assert call(bnn, op, batch={**NONE, **kw}) == want


REFUSED = {
    "rope": [(dict(q=0), ERR_NULL), (dict(k=0), ERR_NULL), (dict(v=0), ERR_NULL), (dict(q_out=0), ERR_NULL), (dict(positions=0), ERR_NULL),
             (dict(turns=0), ERR_NULL), (dict(q=A8), ERR_ALIGN), (dict(src_dtype=1, q=A4), ERR_ALIGN), (dict(q_row=258), ERR_ALIGN),
             (dict(q_out=A8), ERR_ALIGN), (dict(qo_head=68), ERR_ALIGN), (dict(turns=A8), ERR_ALIGN), (dict(q_weight=A4), ERR_ALIGN),
             (dict(positions=A2), ERR_ALIGN), (dict(pos=A2), ERR_ALIGN), (dict(src_dtype=2), ERR_UNSUPPORTED), (dict(rot=12), ERR_UNSUPPORTED),
             (dict(rot=72), ERR_SHAPE), (dict(rot=-8), ERR_SHAPE), (dict(heads=0), ERR_SHAPE), (dict(max_pos=-1), ERR_SHAPE), (dict(k_row=-4), ERR_LD),
             (dict(ld_slots=63), ERR_LD), (dict(eps=-1.0), ERR_UNSUPPORTED), (dict(eps=float("nan")), ERR_UNSUPPORTED)],
    "attn": [(dict(q=0), ERR_NULL), (dict(out=0), ERR_NULL), (dict(q=A8), ERR_ALIGN), (dict(out=A4), ERR_ALIGN), (dict(q_head=60), ERR_ALIGN),
             (dict(o_row=252), ERR_ALIGN), (dict(o_row=-8), ERR_LD), (dict(heads=3), ERR_SHAPE), (dict(heads=0), ERR_SHAPE), (dict(ld_mask=0), ERR_LD),
             (dict(mask=A2), ERR_ALIGN), (dict(out_dtype=2), ERR_UNSUPPORTED), (dict(out_dtype=0), ERR_UNSUPPORTED), (dict(ld_lse=3), ERR_LD),
             (dict(lse=A2), ERR_ALIGN), (dict(scale=float("nan")), ERR_UNSUPPORTED), (dict(scale=float("inf")), ERR_UNSUPPORTED)],
    "score": [(dict(q=0), ERR_NULL), (dict(lse=0), ERR_NULL), (dict(score_in=0), ERR_NULL), (dict(score_out=0), ERR_NULL), (dict(q=A8), ERR_ALIGN),
              (dict(heads=5), ERR_SHAPE), (dict(ld_lse=3), ERR_LD), (dict(ld_slots=63), ERR_LD), (dict(accept=A2), ERR_ALIGN), (dict(ld_accept=0), ERR_LD),
              (dict(ld_mask=-1), ERR_LD), (dict(scale=float("inf")), ERR_UNSUPPORTED)],
    "evict": [(dict(pos_in=0), ERR_NULL), (dict(pos_out=0), ERR_NULL), (dict(score_in=0), ERR_NULL), (dict(score_out=0), ERR_NULL),
              (dict(ctx_out=0), ERR_NULL), (dict(ctx_out=A2), ERR_ALIGN), (dict(score_out=A2), ERR_ALIGN), (dict(budget=-1), ERR_SHAPE),
              (dict(recent=-1), ERR_SHAPE), (dict(ld_slots=63), ERR_LD), (dict(ld_accept=0), ERR_LD)],
}


@pytest.mark.parametrize("op,kw,want", [(op, kw, want) for op, cases in REFUSED.items() for kw, want in cases])
def test_argument_refusals(bnn, op, kw, want):
    assert call(bnn, op, batch=NONE, **kw) == want


def test_workspaces(bnn):
    c, b = fill(bnn._KvCache, CACHE, dict(K=0, V=0)), fill(bnn._KvBatch, BATCH, dict(indptr=0, ctx=0))
    need = bnn.lib().bnn_cache_evict_workspace(ctypes.addressof(c), 2)
    assert need > 0
    assert call(bnn, "evict", workspace=0) == ERR_NULL and call(bnn, "evict", workspace=A8) == ERR_ALIGN
    assert call(bnn, "evict", workspace_bytes=need - 1) == ERR_SHAPE
    assert bnn.lib().bnn_cache_evict_workspace(None, 2) == -1 and bnn.lib().bnn_cache_evict_workspace(ctypes.addressof(c), -1) == -1
    f = bnn.lib().bnn_tree_attention_workspace
    assert f(ctypes.addressof(c), ctypes.addressof(b), 4) >= 0
    assert f(ctypes.addressof(c), ctypes.addressof(b), 3) == -1 and f(None, ctypes.addressof(b), 4) == -1 and f(ctypes.addressof(c), None, 4) == -1
    big = fill(bnn._KvBatch, BATCH, dict(B=1, max_ctx=100000))
    need = f(ctypes.addressof(c), ctypes.addressof(big), 4)
    if need:
        assert call(bnn, "attn", batch=dict(B=1, max_ctx=100000), workspace_bytes=need - 1) == ERR_SHAPE
        assert call(bnn, "attn", batch=dict(B=1, max_ctx=100000), workspace=0) == ERR_NULL


def test_binding_refuses_host_tensors(bnn):
    k = torch.zeros(2, 4, 1, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="HIP device"):
        bnn.KVCache(k, k)
    with pytest.raises(TypeError, match="bfloat16 or torch.float16"):
        bnn.KVCache(k.float(), k.float())


# ---- the rotation table

@pytest.mark.parametrize("kind", ["plain", "linear", "base", "ramp", "bands"])
@pytest.mark.parametrize("rot,base,factor,old", [(128, 1e4, 4.0, 4096), (64, 5e5, 8.0, 8192), (24, 1e4, 1.0, 2048)])
def test_rope_turns(bnn, kind, rot, base, factor, old):
    fast, slow = (32.0, 1.0) if kind != "bands" else (4.0, 1.0)
    got = bnn.rope_turns(1500, rot, base=base, kind=kind, factor=factor, old_ctx=old, beta_fast=fast, beta_slow=slow).double().numpy()
    half, gain = rot // 2, 1.0
    theta = []
    for i in range(half):
        t = base ** (-2 * i / rot)
        turns = old * t / (2 * math.pi)                    # turns of the pair over the first context
        if kind == "linear":
            t /= factor
        elif kind == "base":
            t = (base * factor ** (rot / (rot - 2))) ** (-2 * i / rot)
        elif kind == "bands":
            w = min(max((turns - slow) / (fast - slow), 0.0), 1.0)
            t = t * w + t / factor * (1 - w)
        elif kind == "ramp":
            index = lambda beta: rot * math.log(old / (beta * 2 * math.pi)) / (2 * math.log(base))
            lo, hi = max(math.floor(index(fast)), 0), min(math.ceil(index(slow)), rot - 1)
            w = 1 - min(max((i - lo) / (hi - lo), 0.0), 1.0)
            t = t * w + t / factor * (1 - w)
            gain = 0.1 * math.log(factor) + 1
        theta.append(t)
    angle = np.arange(1500)[:, None] * np.array(theta)[None]
    want = np.concatenate((gain * np.cos(angle), gain * np.sin(angle)), 1)
    # one rounding to fp32, and pow/cos/sin in double off by a few ulp of angles up to 1500
    assert np.abs(got - want).max() <= 2.0 ** -24 * gain + 1500 * 2.0 ** -50
    if kind == "ramp":                                     # both ends of the ramp are there
        assert theta[0] == 1.0 and math.isclose(theta[-1], base ** (-2 * (half - 1) / rot) / factor, rel_tol=1e-12)


def test_rope_turns_refusals(bnn):
    out = torch.empty(64)
    f = lambda max_pos=2, rot=8, base=1e4, kind=0, factor=2.0, old=100.0, fast=32.0, slow=1.0, p=out.data_ptr(): bnn.lib().bnn_rope_turns_host(
        max_pos, rot, base, kind, factor, old, fast, slow, p)
    assert f() == OK and f(max_pos=0) == OK
    assert f(p=None) == ERR_NULL
    assert f(max_pos=-1) == f(rot=7) == f(rot=0) == ERR_SHAPE
    for bad in (dict(base=1.0), dict(base=math.nan), dict(factor=0.5), dict(factor=math.inf), dict(kind=5), dict(kind=-1), dict(kind=3, old=0.0),
                dict(kind=4, fast=1.0), dict(kind=3, slow=0.0), dict(kind=2, rot=2)):
        assert f(**bad) == ERR_UNSUPPORTED, bad


# ---- tree masks

@pytest.mark.parametrize("T", [1, 2, 31, 32, 33, 100])
def test_tree_mask(bnn, T):
    par, seen = ref.random_tree(np.random.default_rng(T), T)
    words = (T + 31) // 32
    for extra in (0, 2):
        assert torch.equal(bnn.tree_mask(par, words + extra), ref.packed(seen, words + extra))
    chain = bnn.tree_mask([i - 1 for i in range(T)])
    assert torch.equal(chain, ref.packed([range(i + 1) for i in range(T)], words))


def test_tree_mask_refusals(bnn):
    for parents in ([0], [-1, 1], [-1, -2], [-1, 0, 3]):
        with pytest.raises(bnn.BnnError) as e:
            bnn.tree_mask(parents)
        assert e.value.status == ERR_UNSUPPORTED
    with pytest.raises(bnn.BnnError) as e:
        bnn.tree_mask([-1] * 33, 1)
    assert e.value.status == ERR_LD
    assert bnn.tree_mask([]).shape == (0, 1)


# ---- the 64-bit references themselves

def test_reference_attention_against_direct_sums():
    rng = np.random.default_rng(1)
    q, k, v = rng.standard_normal((4, 6)), rng.standard_normal((9, 2, 6)), rng.standard_normal((9, 2, 6))
    vis = np.array([1, 1, 0, 1, 1, 0, 1, 1, 1], dtype=bool)
    out, lse, A, S = ref.attention(q, k, v, vis, 0.7)
    for h in range(4):
        e = [math.exp(0.7 * sum(q[h, d] * k[j, h // 2, d] for d in range(6))) if vis[j] else 0.0 for j in range(9)]
        assert math.isclose(lse[h], math.log(sum(e)), rel_tol=1e-13)
        for d in range(6):
            assert math.isclose(out[h, d], sum(e[j] * v[j, h // 2, d] for j in range(9)) / sum(e), rel_tol=1e-11, abs_tol=1e-14)
    out, lse, _, _ = ref.attention(q, k, v, np.zeros(9, dtype=bool), 0.7)
    assert (out == 0).all() and np.isneginf(lse).all()


def test_reference_rope_keeps_lengths_and_relative_positions():
    rng = np.random.default_rng(2)
    x, y = rng.standard_normal((1, 1, 16)), rng.standard_normal((1, 1, 16))
    theta = 10000.0 ** (-np.arange(4) / 4)
    for inter in (False, True):
        dots = []
        for p, r in ((3, 10), (53, 60)):
            a, _ = ref.rope(x, None, 0, np.cos(p * theta)[None], np.sin(p * theta)[None], 8, inter)
            b, _ = ref.rope(y, None, 0, np.cos(r * theta)[None], np.sin(r * theta)[None], 8, inter)
            assert math.isclose((a * a).sum(), (x * x).sum(), rel_tol=1e-12) and (a[..., 8:] == x[..., 8:]).all()
            dots.append(float((a * b).sum()))
        assert math.isclose(dots[0], dots[1], rel_tol=1e-9)


def test_reference_evict_by_hand():
    pos, score = np.arange(8), np.array([5.0, 1, 9, 0, 9, 2, 7, 3])
    keep, source = ref.evict(6, 2, [False, True], 4, 0, pos, score)     # slot 6 is rejected: of 0-5 and 7 stay 0, 2, 4, 7
    assert keep == 4 and source.tolist() == [0, 4, 2, 7]
    keep, source = ref.evict(6, 2, [True, True], 4, 2, pos, score)      # 6 and 7 are recent; then 2 and 4
    assert source.tolist() == [4, 6, 2, 7]
    keep, source = ref.evict(6, 2, [False, False], 100, 2, pos, score)
    assert keep == 6 and source.tolist() == list(range(6))
    assert ref.evict(3, 0, None, 2, 0, pos, np.array([1.0, 1.0, np.nan]))[1].tolist() == [0, 1]
