"""GPU checks of the calls over the paged key/value cache against their
definitions in 64 bits: norm + rotation + append, tree attention, the
attention-weight sums and the eviction.

Bounds.  A 16-bit output is rounded once (u = half an ulp as a ratio); with a
16-bit attention output each weight is rounded to that type too.  A product
<q, k> of D terms in fp32 is off by at most (D + 2) 2^-24 sum |q k|, which
the exponent turns into a relative error ds = (D + 2) 2^-24 scale sum |q k| +
8 2^-24 max |s| of a weight; sums over n slots add n 2^-24."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import cache_ref as ref
from gpu_util import require_gpu, banner

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float16


@pytest.fixture(scope="module")
def bnn():
    require_gpu()
    import xnor_popcount_gemm_amd as m
    m.lib()
    return m


def cuda_i32(x):
    return torch.tensor(x, dtype=torch.int32).cuda()


def strided(x, pad):
    """x on the GPU as a view with `pad` spare elements between rows (NaN)."""
    if not pad:
        return x.cuda()
    big = torch.full((*x.shape[:-2], x.shape[-2] + 1, x.shape[-1] + pad), float("nan"), dtype=x.dtype, device="cuda")
    view = big[..., : x.shape[-2], : x.shape[-1]]
    view.copy_(x)
    return view


# ---- norm, rotation, append

ROPE = [
    # kind, src, heads, kv, dim, rot, interleaved, norm, ctx, nodes, page, order, pad
    (BF, torch.float32, 32, 8, 128, 128, False, True, [100], [1], 16, "token", 0),
    (BF, torch.float32, 4, 1, 64, 32, True, True, [0, 5, 17], [3, 0, 9], 4, "head", 8),
    (FP, FP, 6, 3, 96, 48, False, False, [31, 1], [33, 2], 24, "token", 8),
    (FP, torch.float32, 5, 5, 256, 256, True, True, [7], [70], 1, "token", 0),
    (BF, BF, 3, 3, 96, 8, False, True, [2, 3], [1, 1], 64, "head", 0),
    (BF, BF, 8, 2, 64, 0, False, True, [9], [4], 3, "token", 0),
]


@pytest.mark.parametrize("case", ROPE, ids=range(len(ROPE)))
def test_rope_append(bnn, case):
    kind, src, heads, kv, dim, rot, inter, norm, ctx, nodes, page, order, pad = case
    banner(f"qk_norm_rope {case}")
    rng = np.random.default_rng(11)
    B, rows = len(ctx), sum(nodes)
    cache = ref.Paged(rng, B, max(c + t for c, t in zip(ctx, nodes)) + 5, page, kv, dim, kind, order)
    q, k, v = (torch.from_numpy(rng.standard_normal((rows, n, dim)) * 3).to(src) for n in (heads, kv, kv))
    wq, wk = (torch.from_numpy(1 + 0.2 * rng.standard_normal(dim)).float() for _ in range(2)) if norm else (None, None)
    turns = bnn.rope_turns(200, rot, kind="linear", factor=2.0) if rot else None
    positions = rng.integers(0, 200, rows).astype(np.int32)
    pos = torch.full((B, kv, cache.slots + 3), -7, dtype=torch.int32, device="cuda")
    score = torch.full((B, kv, cache.slots + 3), 5.0, device="cuda")
    dc = cache.device(bnn, pos, score)
    indptr = np.concatenate(([0], np.cumsum(nodes)))
    got = bnn.qk_norm_rope(strided(q, pad), strided(k, pad), strided(v, pad), dc, cuda_i32(indptr), cuda_i32(ctx),
                           torch.from_numpy(positions).cuda(), None if turns is None else turns.cuda(),
                           q_weight=None if wq is None else wq.cuda(), k_weight=None if wk is None else wk.cuda(),
                           eps=1e-5, interleaved=inter)
    torch.cuda.synchronize()
    t = turns.double().numpy()[positions] if rot else np.zeros((rows, 0))
    want = {}
    for name, x, w in (("q", q, wq), ("k", k, wk)):
        want[name] = ref.rope(x.double().numpy(), None if w is None else w.double().numpy(), 1e-5, t[:, : rot // 2], t[:, rot // 2:], rot, inter)

    def check(x, name, sel=slice(None)):
        y, mag = want[name][0][sel], want[name][1][sel]
        err = np.abs(x - y)
        bound = ref.U[kind] * np.abs(y) + (dim + 16) * ref.E32 * mag + 2.0 ** -25
        assert (err <= bound).all(), (name, float((err / bound).max()))

    check(got.double().cpu().numpy(), "q")
    cache.K, cache.V = cache.dK.cpu(), cache.dV.cpu()
    used = torch.zeros(cache.K.shape[:2], dtype=torch.bool)
    pos, score = pos.cpu().numpy(), score.cpu().numpy()
    for b in range(B):
        rows_b = slice(indptr[b], indptr[b + 1])
        s = ctx[b] + np.arange(nodes[b])
        check(cache.get("K", b, s), "k", rows_b)
        assert torch.equal(cache.V[cache.at(b, s)], v[rows_b].to(kind))
        used[cache.at(b, s)] = True
        assert (pos[b][:, s] == positions[rows_b]).all() and (score[b][:, s] == 0).all()
        rest = np.setdiff1d(np.arange(pos.shape[2]), s)
        assert (pos[b][:, rest] == -7).all() and (score[b][:, rest] == 5).all()
    assert cache.K[~used].isnan().all() and cache.V[~used].isnan().all()


def test_rope_bad_tokens(bnn):
    """A position outside the table gives NaN; rows past the last sequence, a
    slot past the capacity and a page outside the cache are not written."""
    banner("qk_norm_rope out of range")
    rng = np.random.default_rng(3)
    cache = ref.Paged(rng, 2, 8, 4, 2, 64, BF)
    cache.table[1, 1] = 999
    dc = cache.device(bnn)
    q, k, v = (torch.randn(7, n, 64) for n in (2, 2, 2))
    out = torch.full((7, 2, 64), 3.0, dtype=BF, device="cuda")
    bnn.qk_norm_rope(q.cuda(), k.cuda(), v.cuda(), dc, cuda_i32([0, 3, 6]), cuda_i32([6, 3]), cuda_i32([0, 10, -1, 0, 1, 2, 3]),
                     bnn.rope_turns(10, 32).cuda(), q_out=out)
    out, K = out.cpu(), cache.dK.cpu()
    assert out[1:3, :, :32].isnan().all() and not out[1:3, :, 32:].isnan().any() and not out[0].isnan().any()
    assert (out[6] == 3).all()
    written = ~K.isnan().all(-1).all(-1)
    want = torch.zeros_like(written)
    want[cache.table[0, 1].long(), 2:4] = True    # slots 6, 7 of sequence 0; 8 does not fit
    want[cache.table[1, 0].long(), 3] = True      # slot 3 of sequence 1; 4 and 5 have no page
    assert torch.equal(written, want)


# ---- attention

ATTN = [
    # kind, out, heads, kv, dim, ctx, nodes, page, order, tree, table
    (BF, torch.float32, 32, 8, 128, [1], [1], 16, "token", False, True),
    (BF, BF, 8, 1, 128, [0, 1, 63, 64, 65, 500], [1, 1, 1, 1, 0, 1], 16, "token", False, True),
    (FP, FP, 6, 6, 64, [33, 0, 200], [13, 5, 16], 24, "head", True, True),
    (BF, torch.float32, 10, 2, 96, [129, 31], [7, 40], 1, "token", True, True),
    (FP, torch.float32, 8, 2, 256, [300, 17], [3, 33], 64, "head", True, True),
    (BF, BF, 28, 4, 128, [1000, 40], [63, 64], 16, "token", True, True),
    (BF, BF, 16, 4, 64, [77, 513], [130, 70], 128, "token", False, True),
    (FP, FP, 4, 1, 96, [257], [65], 33, "token", True, True),
    (BF, BF, 2, 1, 256, [5, 700], [90, 100], 7, "token", False, True),
    (BF, torch.float32, 8, 8, 128, [3000, 1], [2, 2], 4096, "head", True, False),
    (FP, FP, 16, 2, 128, [6000], [1], 256, "token", False, True),
    (FP, torch.float32, 40, 8, 128, [0, 0], [100, 1], 32, "head", True, True),
]


def make_attention(case, seed=5, q_by=2.0):
    kind, out, heads, kv, dim, ctx, nodes, page, order, tree, table = case
    rng = np.random.default_rng(seed)
    B, rows = len(ctx), sum(nodes)
    cache = ref.Paged(rng, B, max(c + t for c, t in zip(ctx, nodes)) + 3, page, kv, dim, kind, order, table)
    for b in range(B):
        s = np.arange(ctx[b] + nodes[b])
        for w in "KV":
            cache.put(w, b, s, rng.standard_normal((len(s), kv, dim)))
    q = torch.from_numpy(rng.standard_normal((rows, heads, dim)) * q_by).to(kind)
    seen = []
    for t in nodes:
        seen += ref.random_tree(rng, t)[1]
    words = max(1, -(-max(nodes) // 32))
    return rng, cache, q, ref.packed(seen, words) if tree else None, seen if tree else None


def check_attention(case, cache, q, seen, got, lse, scale, what=""):
    kind, out, heads, kv, dim, ctx, nodes = case[:7]
    got, lse = got.double().cpu().numpy(), lse.double().cpu().numpy()
    u = ref.U[out] + (ref.U[out] if out != torch.float32 else 2.0 ** -22)
    row = 0
    for b, (c, t) in enumerate(zip(ctx, nodes)):
        k, v = (cache.get(w, b, np.arange(c + t)) for w in "KV")
        for i in range(t):
            vis = ref.sees(c, t, i, None if seen is None else np.isin(np.arange(t), list(seen[row])))
            y, l, A, S = ref.attention(q[row].double().numpy(), k, v, vis, scale)
            n = int(vis.sum())
            empty = np.isneginf(l)
            ds = (dim + 10) * ref.E32 * S
            assert np.array_equal(np.isneginf(lse[row]), empty), (what, b, i)
            if not empty.all():
                bl = ds + (n + 8) * ref.E32 + 8 * ref.E32 * np.abs(l)
                assert (np.abs(lse[row] - l) <= bl).all(), (what, "lse", b, i, float((np.abs(lse[row] - l) / bl).max()))
            bound = u * A + (2 * ds + 2 * n * ref.E32)[:, None] * A + 2.0 ** -26
            err = np.abs(got[row] - y)
            assert (err <= bound).all(), (what, "out", b, i, float((err / bound).max()))
            row += 1


@pytest.mark.parametrize("case", ATTN, ids=range(len(ATTN)))
def test_tree_attention(bnn, case):
    kind, out, heads, kv, dim, ctx, nodes, page, order, tree, table = case
    banner(f"tree_attention {case}")
    rng, cache, q, mask, seen = make_attention(case)
    dc = cache.device(bnn)
    indptr = cuda_i32(np.concatenate(([0], np.cumsum(nodes))))
    scale = 1.1 * dim ** -0.5
    dq = strided(q, 8)
    dm = None if mask is None else mask.cuda()
    got, lse = bnn.tree_attention(dq, dc, indptr, cuda_i32(ctx), max_nodes=max(nodes), max_ctx=max(ctx), mask=dm, scale=scale, out_dtype=out)
    torch.cuda.synchronize()
    check_attention(case, cache, q, seen, got, lse, scale)
    # bounds that are too wide, a ctx past the bound, another stream, a strided output: the same function
    wide, lse2 = bnn.tree_attention(dq, dc, indptr, cuda_i32(ctx), max_nodes=max(nodes) + 40, max_ctx=5 * max(ctx) + 999, mask=dm, scale=scale, out_dtype=out)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        o3 = torch.full((q.shape[0], heads + 1, dim + 8), 9.0, dtype=out, device="cuda")
        tight, lse3 = bnn.tree_attention(dq, dc, indptr, cuda_i32(ctx), max_nodes=max(nodes), max_ctx=0, mask=dm, scale=scale, out=o3[:, :heads, :dim])
    s.synchronize()
    torch.cuda.synchronize()
    check_attention(case, cache, q, seen, wide, lse2, scale, "wide bounds")
    check_attention(case, cache, q, seen, tight, lse3, scale, "tight bounds")
    assert (o3[:, heads:] == 9).all() and (o3[..., dim:] == 9).all()


@pytest.mark.parametrize("case", [ATTN[i] for i in (2, 3, 5, 7)], ids=(2, 3, 5, 7))
def test_attention_rows_that_see_nothing_and_poisoned_drafts(bnn, case):
    """Masked tokens hold NaN and infinities, some rows see nothing at all;
    a row that sees a poisoned token is poisoned where the definition says."""
    kind, out, heads, kv, dim, ctx, nodes, page, order, tree, table = case
    banner(f"tree_attention poisoned {case}")
    rng, cache, q, mask, seen = make_attention(case, seed=8)
    ctx = list(ctx)
    ctx[0] = 0                                   # sequence 0 has drafts alone
    seen[0] = set()                              # and its first row sees nothing
    T, first = nodes[-1], sum(nodes[:-1])
    b, c = len(ctx) - 1, ctx[-1]
    poison = {1: float("nan"), 2: float("inf"), T - 1: float("-inf")}
    for j, x in poison.items():
        cache.put("V", b, [c + j], np.full((1, kv, dim), x))
    cache.put("K", b, [c + 1], np.full((1, kv, dim), np.nan))
    only = {first + 2: {0, 2}, first + T - 1: {0, 2, T - 1}}   # +inf; +inf and -inf
    for i in range(T):
        seen[first + i] = only.get(first + i, set(seen[first + i]) - set(poison))
    case = case[:5] + (ctx,) + case[6:]
    mask = ref.packed(seen, mask.shape[1]).cuda()
    dc = cache.device(bnn)
    scale = dim ** -0.5
    got, lse = bnn.tree_attention(q.cuda(), dc, cuda_i32(np.concatenate(([0], np.cumsum(nodes)))), cuda_i32(ctx), max_nodes=max(nodes),
                                  max_ctx=max(case[5]), mask=mask, scale=scale, out_dtype=out)
    torch.cuda.synchronize()
    g = got.float().cpu()
    assert (g[first + 2] == float("inf")).all(), "a row that sees +inf"
    assert g[first + T - 1].isnan().all(), "a row that sees +inf and -inf"
    for r in only:                               # the others by value
        got[r], seen[r] = 0, set()
        lse[r] = float("-inf")
    # rows `only` see committed slots too: compare all other rows
    keep = [r for r in range(sum(nodes)) if r not in only]
    got, lse = got.double().cpu().numpy(), lse.double().cpu().numpy()
    row = 0
    u = ref.U[out] + (ref.U[out] if out != torch.float32 else 2.0 ** -22)
    for b, (c, t) in enumerate(zip(ctx, nodes)):
        k, v = (cache.get(w, b, np.arange(c + t)) for w in "KV")
        for i in range(t):
            if row in keep:
                vis = ref.sees(c, t, i, np.isin(np.arange(t), list(seen[row])))
                y, l, A, S = ref.attention(q[row].double().numpy(), k, v, vis, scale)
                assert np.array_equal(np.isneginf(lse[row]), np.isneginf(l)), (b, i)
                bound = u * A + (2 * (dim + 10) * ref.E32 * S + 2 * (c + t) * ref.E32)[:, None] * A + 2.0 ** -26
                assert (np.abs(got[row] - y) <= bound).all(), (b, i)
            row += 1
    assert np.isneginf(lse[0]).all() and (got[0] == 0).all()


@pytest.mark.parametrize("T,heads,kv", [(1, 8, 2), (9, 8, 4), (40, 8, 2)])
def test_attention_extreme_logits(bnn, T, heads, kv):
    """Logits of hundreds, a maximum that comes last, and equal logits."""
    banner(f"tree_attention extreme logits T={T}")
    case = (BF, torch.float32, heads, kv, 128, [900], [T], 16, "token", True, True)
    rng, cache, q, mask, seen = make_attention(case, seed=21, q_by=40.0)
    n = 900 + T
    ramp = np.sign(q[0].double().numpy()[:: heads // kv])[None] * np.linspace(0.0, 1.5, n)[:, None, None]   # grows along the slots for row 0
    cache.put("K", 0, np.arange(n), ramp)
    dc = cache.device(bnn)
    got, lse = bnn.tree_attention(q.cuda(), dc, cuda_i32([0, T]), cuda_i32([900]), max_nodes=T, max_ctx=900, mask=mask.cuda(), scale=0.09, out_dtype=torch.float32)
    torch.cuda.synchronize()
    check_attention(case, cache, q, seen, got, lse, 0.09)
    cache.put("K", 0, np.arange(n), np.zeros((n, kv, 128)))
    dc = cache.device(bnn)
    got, lse = bnn.tree_attention(q.cuda(), dc, cuda_i32([0, T]), cuda_i32([900]), max_nodes=T, max_ctx=900, mask=mask.cuda(), scale=0.09, out_dtype=torch.float32)
    check_attention(case, cache, q, seen, got, lse, 0.09)


@pytest.mark.parametrize("scale", [0.0, -0.07])
@pytest.mark.parametrize("T,heads,kv", [(1, 4, 1), (11, 4, 2), (50, 8, 2)])
def test_attention_zero_and_negative_scale(bnn, scale, T, heads, kv):
    banner(f"tree_attention scale {scale} T={T}")
    case = (BF, torch.float32, heads, kv, 64, [210], [T], 16, "token", True, True)
    rng, cache, q, mask, seen = make_attention(case, seed=31)
    got, lse = bnn.tree_attention(q.cuda(), cache.device(bnn), cuda_i32([0, T]), cuda_i32([210]), max_nodes=T, max_ctx=210, mask=mask.cuda(), scale=scale,
                                  out_dtype=torch.float32)
    out, want = got.double().cpu().numpy(), lse.double().cpu().numpy()
    k, v = (cache.get(w, 0, np.arange(210 + T)) for w in "KV")
    for i in range(T):
        y, l, A, S = ref.attention(q[i].double().numpy(), k, v, ref.sees(210, T, i, np.isin(np.arange(T), list(seen[i]))), scale)
        ds = (64 + 10) * ref.E32 * np.abs(S)
        assert (np.abs(want[i] - l) <= ds + (210 + T + 8) * ref.E32 + 8 * ref.E32 * np.abs(l)).all()
        assert (np.abs(out[i] - y) <= (2.0 ** -22 + 2.0 ** -24 + 2 * ds + 2 * (210 + T) * ref.E32)[:, None] * A + 2.0 ** -26).all()


@pytest.mark.parametrize("T", [1, 40])
def test_attention_missing_page(bnn, T):
    """A table entry that names no page reads as rows of zeros."""
    banner(f"tree_attention missing page T={T}")
    case = (FP, torch.float32, 8, 2, 128, [200], [T], 16, "token", True, True)
    rng, cache, q, mask, seen = make_attention(case, seed=32)
    for w in "KV":
        cache.put(w, 0, np.arange(48, 64), np.zeros((16, 2, 128)))
    args = dict(max_nodes=T, max_ctx=200, mask=mask.cuda(), out_dtype=torch.float32)
    want, l0 = bnn.tree_attention(q.cuda(), cache.device(bnn), cuda_i32([0, T]), cuda_i32([200]), **args)
    for bad in (-1, 1 << 30):
        cache.table[0, 3] = bad
        dc = cache.device(bnn, score=torch.zeros((1, 2, cache.slots), device="cuda"))
        got, l1 = bnn.tree_attention(q.cuda(), dc, cuda_i32([0, T]), cuda_i32([200]), **args)
        assert torch.equal(got, want) and torch.equal(l0, l1)
        assert bnn.cache_score_add(q.cuda(), l1, dc, cuda_i32([0, T]), cuda_i32([200]), max_nodes=T, max_ctx=200, mask=mask.cuda()).isfinite().all()


def test_many_sequences(bnn):
    """130 short sequences, some without committed and some without new tokens:
    every call's way from a row or a share of the work to its sequence."""
    banner("130 sequences")
    rng = np.random.default_rng(33)
    B, heads, kv, dim = 130, 4, 2, 64
    ctx, nodes = rng.integers(0, 70, B), rng.integers(0, 4, B)
    ctx[[0, 64, 129]], nodes[[0, 63, 65, 128]] = 0, 0
    case = (BF, torch.float32, heads, kv, dim, ctx.tolist(), nodes.tolist(), 8, "token", False, True)
    _, cache, q, _, _ = make_attention(case, seed=34)
    rows = int(nodes.sum())
    score = torch.zeros((B, kv, cache.slots), device="cuda")
    pos = torch.full((B, kv, cache.slots), -1, dtype=torch.int32, device="cuda")
    dc = cache.device(bnn, pos, score)
    indptr, dctx = cuda_i32(np.concatenate(([0], np.cumsum(nodes)))), cuda_i32(ctx)
    k, v = torch.from_numpy(rng.standard_normal((2, rows, kv, dim))).float()
    qr = bnn.qk_norm_rope(q.float().cuda(), k.cuda(), v.cuda(), dc, indptr, dctx, cuda_i32(range(rows)), None)
    assert torch.equal(qr.cpu(), q)
    starts = np.concatenate(([0], np.cumsum(nodes)))
    for b in range(B):
        s = ctx[b] + np.arange(nodes[b])
        rows_b = slice(starts[b], starts[b + 1])
        assert torch.equal(pos.cpu()[b][:, s], torch.arange(rows, dtype=torch.int32)[rows_b].expand(kv, -1))
        cache.put("K", b, s, k[rows_b])
        cache.put("V", b, s, v[rows_b])
    args = dict(max_nodes=3, max_ctx=70)
    out, lse = bnn.tree_attention(qr, dc, indptr, dctx, out_dtype=torch.float32, **args)
    torch.cuda.synchronize()
    check_attention(case, cache, q, None, out, lse, dim ** -0.5)
    # the weights of a row add up to the heads of its group, so the sums count the rows
    total = bnn.cache_score_add(qr, lse, dc, indptr, dctx, **args).double().sum(-1).cpu().numpy()
    assert np.allclose(total, nodes[:, None] * (heads // kv) * np.ones((1, kv)), rtol=2e-5, atol=0)
    got = bnn.cache_evict(dc, indptr, dctx, budget=50, recent=0, **args)
    assert np.array_equal(got.cpu().numpy(), np.minimum(ctx + nodes, 50))


def test_attention_far_pages(bnn):
    """Rows that lie past 2^32 bytes of the cache's start."""
    banner("tree_attention far pages")
    page, kv, dim, pages = 128, 8, 128, 16500          # 4.3 GB each of K and V
    K = torch.empty((pages, page, kv, dim), dtype=FP, device="cuda")
    V = torch.empty_like(K)
    table = torch.tensor([[16499, 3, 16450]], dtype=torch.int32, device="cuda")
    near = torch.randn((3, page, kv, dim), device="cuda").to(FP), torch.randn((3, page, kv, dim), device="cuda").to(FP)
    K[table[0].long()], V[table[0].long()] = near
    q = torch.randn((2, 16, dim), device="cuda").to(FP)
    args = dict(max_nodes=2, max_ctx=300)
    indptr, ctx = cuda_i32([0, 2]), cuda_i32([300])
    far, lse = bnn.tree_attention(q, bnn.KVCache(K, V, table), indptr, ctx, **args)
    want, lse2 = bnn.tree_attention(q, bnn.KVCache(*near, cuda_i32([[0, 1, 2]])), indptr, ctx, **args)
    sc = torch.zeros((1, kv, 3 * page), device="cuda")
    s1 = bnn.cache_score_add(q, lse, bnn.KVCache(K, V, table, score=sc.clone()), indptr, ctx, **args)
    s2 = bnn.cache_score_add(q, lse, bnn.KVCache(*near, cuda_i32([[0, 1, 2]]), score=sc.clone()), indptr, ctx, **args)
    torch.cuda.synchronize()
    assert torch.equal(far, want) and torch.equal(lse, lse2) and torch.equal(s1, s2) and float(s1.sum()) > 0


# ---- running sums of attention weight

@pytest.mark.parametrize("case", [ATTN[i] for i in (0, 1, 2, 3, 4, 5, 6, 7, 9, 11)], ids=(0, 1, 2, 3, 4, 5, 6, 7, 9, 11))
def test_score_add(bnn, case):
    kind, out, heads, kv, dim, ctx, nodes, page, order, tree, table = case
    banner(f"cache_score_add {case}")
    rng, cache, q, mask, seen = make_attention(case, seed=6, q_by=1.0)
    B, rows, scale = len(ctx), sum(nodes), dim ** -0.5
    score = torch.from_numpy(rng.random((B, kv, cache.slots + 2))).float()
    lse = torch.from_numpy(rng.standard_normal((rows, heads)) + 3).float()
    lse[0, 0] = float("-inf")                   # a row that saw nothing adds nothing
    take = [[i for i in range(t) if rng.random() < 0.4 or i == 0] for t in nodes]
    words = max(1, -(-max(nodes) // 32))
    indptr = cuda_i32(np.concatenate(([0], np.cumsum(nodes))))
    g = heads // kv
    for accept, taken in ((ref.packed(take, words), take), (None, [list(range(t)) for t in nodes])):
        dc = cache.device(bnn, score=score.cuda())
        res = torch.full(score.shape, 77.0, device="cuda")
        got = bnn.cache_score_add(strided(q, 8), lse.cuda(), dc, indptr, cuda_i32(ctx), max_nodes=max(nodes), max_ctx=max(ctx),
                                  mask=None if mask is None else mask.cuda(), accept=None if accept is None else accept.cuda(), scale=scale, score_out=res)
        again = bnn.cache_score_add(strided(q, 8), lse.cuda(), dc, indptr, cuda_i32(ctx), max_nodes=max(nodes) + 9, max_ctx=0,
                                    mask=None if mask is None else mask.cuda(), accept=None if accept is None else accept.cuda(), scale=scale)
        torch.cuda.synchronize()
        got, again = got.double().cpu().numpy(), again.double().cpu().numpy()
        row = 0
        for b, (c, t) in enumerate(zip(ctx, nodes)):
            k = cache.get("K", b, np.arange(c + t))
            add, tol = np.zeros((kv, c + t)), np.zeros((kv, c + t))
            for i in range(t):
                if i in taken[b]:
                    vis = ref.sees(c, t, i, None if seen is None else np.isin(np.arange(t), list(seen[row])))
                    for h in range(heads):
                        l = float(lse[row, h])
                        if np.isneginf(l):
                            continue
                        x = k[:, h // g] @ q[row, h].double().numpy() * scale
                        S = np.abs(k[:, h // g]) @ np.abs(q[row, h].double().numpy()) * scale
                        w = np.where(vis, np.exp(x - l), 0)
                        add[h // g] += w
                        tol[h // g] += w * ((dim + 10) * S + 8 * np.abs(x) + 8 * abs(l) + 8 + len(taken[b]) * g) * ref.E32
                row += 1
            want = score[b, :, : c + t].double().numpy() + add
            bound = tol + 2 * ref.E32 * np.abs(want)
            for x in (got, again):
                err = np.abs(x[b, :, : c + t] - want)
                assert (err <= bound).all(), (b, float((err / bound).max()))
            for x in (got, again):
                assert np.array_equal(x[b, :, c + t:], score[b, :, c + t:].double().numpy())


# ---- eviction

EVICT = [
    # ctx, nodes, accepted share, budget, recent, page, order
    ([100], [1], 1.0, 100, 10, 16, "token"),
    ([700, 0, 64, 1], [5, 3, 0, 1], 0.5, 64, 16, 4, "head"),
    ([2500, 1030], [31, 2], 0.3, 1024, 0, 64, "token"),
    ([40, 50], [7, 33], 0.5, 1000, 5, 8, "token"),         # nothing to evict: drafts out only
    ([300], [4], 1.0, 0, 3, 16, "token"),                  # nothing kept
    ([5000], [1], 1.0, 1, 0, 256, "head"),
    ([1500], [3], 0.0, 700, 2000, 16, "token"),            # every token recent: the lowest slots
    ([9000, 33], [64, 64], 0.1, 4096, 512, 128, "token"),
    ([40000], [1], 1.0, 5000, 100, 64, "token"),
]


@pytest.mark.parametrize("inplace", (False, True))
@pytest.mark.parametrize("case", EVICT, ids=range(len(EVICT)))
def test_evict(bnn, case, inplace):
    ctx, nodes, share, budget, recent, page, order = case
    banner(f"cache_evict {case} inplace={inplace}")
    rng = np.random.default_rng(17)
    B, kv, dim = len(ctx), 3, 64
    cache = ref.Paged(rng, B, max(c + t for c, t in zip(ctx, nodes)) + 2, page, kv, dim, BF, order)
    pos = np.full((B, kv, cache.slots + 1), -3, dtype=np.int32)
    score = np.full((B, kv, cache.slots + 1), 2.5, dtype=np.float32)
    take = [[i for i in range(t) if share == 1.0 or rng.random() < share] for t in nodes]
    for b in range(B):
        n = ctx[b] + nodes[b]
        for w in "KV":
            cache.put(w, b, np.arange(n), rng.standard_normal((n, kv, dim)))
        for h in range(kv):
            pos[b, h, :n] = rng.permutation(n) * 2
            x = rng.standard_normal(n).astype(np.float32) ** 2
            x[rng.random(n) < 0.2] = 0.0                              # ties
            x[rng.random(n) < 0.1] = rng.choice(np.array([-0.0, 1.0, np.inf, -np.inf, np.nan, 1e-42], dtype=np.float32))
            score[b, h, :n] = x
    before = cache.K.clone(), cache.V.clone()
    dpos, dscore, dctx = torch.from_numpy(pos.copy()).cuda(), torch.from_numpy(score.copy()).cuda(), cuda_i32(ctx)
    dc = cache.device(bnn, dpos, dscore)
    words = max(1, -(-max(nodes) // 32))
    kw = {} if inplace else dict(pos_out=torch.full_like(dpos, -9), score_out=torch.full_like(dscore, -9.0), ctx_out=torch.full_like(dctx, -9))
    for _ in range(1 if inplace else 2):         # with other outputs than inputs a second call changes nothing
        got = bnn.cache_evict(dc, cuda_i32(np.concatenate(([0], np.cumsum(nodes)))), dctx, budget=budget, recent=recent, max_nodes=max(nodes),
                              max_ctx=max(ctx), accept=ref.packed(take, words).cuda(), **kw)
    torch.cuda.synchronize()
    got = got.cpu().numpy()
    K, V = cache.dK.cpu(), cache.dV.cpu()
    pos2, score2 = (dpos, dscore) if inplace else (kw["pos_out"], kw["score_out"])
    pos2, score2 = pos2.cpu().numpy(), score2.cpu().numpy()
    wantK, wantV = before[0].clone(), before[1].clone()
    for b in range(B):
        n = ctx[b] + nodes[b]
        for h in range(kv):
            keep, source = ref.evict(ctx[b], nodes[b], [i in take[b] for i in range(nodes[b])], budget, recent, pos[b, h], score[b, h])
            assert got[b] == keep
            assert np.array_equal(pos2[b, h, :keep], pos[b, h, source]) and (pos2[b, h, keep:n] == -1).all()
            assert np.array_equal(score2[b, h, :keep].view(np.int32), score[b, h, source].view(np.int32)) and (score2[b, h, keep:n] == 0).all()
            if not inplace:
                assert (pos2[b, h, n:] == -9).all() and (score2[b, h, n:] == -9).all()
            if keep:
                p, o = cache.at(b, np.arange(keep))
                ps, os_ = cache.at(b, source)
                wantK[p, o, h], wantV[p, o, h] = before[0][ps, os_, h], before[1][ps, os_, h]
    same = lambda x, y: torch.equal(x.contiguous().view(torch.int16), y.contiguous().view(torch.int16))
    assert same(K, wantK) and same(V, wantV)


# ---- a step as it is used, and in a graph

def test_step_in_a_graph(bnn):
    """Append, attend, sum and evict, captured once and replayed: every replay
    gives what the same eager calls give on a copy."""
    banner("cache step in a graph")
    rng = np.random.default_rng(2)
    B, kv, heads, dim, page, T = 3, 2, 8, 128, 16, 5
    budget = 40
    def fresh():
        cache = ref.Paged(np.random.default_rng(4), B, budget + T + 3, page, kv, dim, BF)
        cache.K.fill_(0), cache.V.fill_(0)
        pos = torch.full((B, kv, cache.slots), -1, dtype=torch.int32, device="cuda")
        score = torch.zeros((B, kv, cache.slots), device="cuda")
        return cache, cache.device(bnn, pos, score), torch.zeros(B, dtype=torch.int32, device="cuda")
    parents, seen = ref.random_tree(rng, T)
    mask = torch.cat([bnn.tree_mask(parents)] * B).cuda()
    accept = ref.packed([[0], [0, T - 1], range(T)], 1).cuda()
    indptr = cuda_i32([T * i for i in range(B + 1)])
    turns = bnn.rope_turns(4096, dim).cuda()
    qkv = torch.empty((B * T, (heads + 2 * kv) * dim), device="cuda")
    positions = torch.empty(B * T, dtype=torch.int32, device="cuda")
    q, k, v = (x.unflatten(1, (-1, dim)) for x in qkv.split([heads * dim, kv * dim, kv * dim], 1))

    def step(dc, ctx, ws):
        qr = bnn.qk_norm_rope(q, k, v, dc, indptr, ctx, positions, turns)
        out, lse = bnn.tree_attention(qr, dc, indptr, ctx, max_nodes=T, max_ctx=budget, mask=mask, out_dtype=torch.float32, workspace=ws[0])
        bnn.cache_score_add(qr, lse, dc, indptr, ctx, max_nodes=T, max_ctx=budget, mask=mask, accept=accept)
        bnn.cache_evict(dc, indptr, ctx, budget=budget, recent=8, max_nodes=T, max_ctx=budget, accept=accept, workspace=ws[1])
        return out, lse

    inputs = [(torch.randn_like(qkv), torch.randint(0, 4000, (B * T,), dtype=torch.int32, device="cuda")) for _ in range(14)]
    results = []
    for graphed in (False, True):
        host, dc, ctx = fresh()
        ws = bnn.tree_attention_workspace(dc, B * T, heads, T, budget), bnn.cache_evict_workspace(dc)
        if graphed:
            qkv.copy_(inputs[0][0]), positions.copy_(inputs[0][1])
            torch.cuda.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                captured = step(dc, ctx, ws)
        outs = []
        for x, p in inputs:
            qkv.copy_(x), positions.copy_(p)
            if graphed:
                graph.replay()
                outs.append([t.clone() for t in captured] + [ctx.clone()])
            else:
                outs.append(list(step(dc, ctx, ws)) + [ctx.clone()])
            torch.cuda.synchronize()
        results.append((outs, dc.pos.clone(), dc.score.clone(), host.dK.clone(), host.dV.clone()))
    eager, graphed = results
    for a, b in zip(eager[0], graphed[0]):
        assert all(torch.equal(x, y) for x, y in zip(a, b))
    assert all(torch.equal(x, y) for x, y in zip(eager[1:], graphed[1:]))
    assert eager[0][-1][2].tolist() == [14, 28, 40]


def test_example_path(bnn):
    """The example's path: ternary projections around the cache calls.  Its
    last step's attention is checked against the definition on what the cache
    held, and the cache against what it must hold."""
    banner("examples/decode_tree.py")
    import os
    import sys
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import decode_tree
    block, y, length = decode_tree.run(steps=30, sequences=3, hidden=256, heads=4, kv_heads=2, dim=64, budget=60, recent=16, nodes=9)
    torch.cuda.synchronize()
    assert y.shape == (27, 256) and y.isfinite().all()
    ctx, pos = block.ctx.cpu().numpy(), block.cache.pos.cpu().numpy()
    for b in range(3):
        assert length[b] > 60 and ctx[b] == 60
        for h in range(2):
            held = pos[b, h, :60]
            assert len(set(held.tolist())) == 60 and held.min() >= 0 and held.max() == length[b] - 1
            assert set(range(length[b] - 16, length[b])) <= set(held.tolist())     # the recent positions stay
            assert (pos[b, h, 60:] == -1).all()
    # one more step, plain decoding: a token per sequence over what is in the cache
    q = torch.randn((3, 4, 64), device="cuda").to(torch.bfloat16)
    indptr = cuda_i32([0, 1, 2, 3])
    k = torch.randn((3, 2, 64), device="cuda")
    qr = bnn.qk_norm_rope(q.float(), k, k, block.cache, indptr, block.ctx, cuda_i32(length), block.turns)
    out, lse = bnn.tree_attention(qr, block.cache, indptr, block.ctx, max_nodes=1, max_ctx=60, out_dtype=torch.float32)
    torch.cuda.synchronize()
    paged = ref.Paged.__new__(ref.Paged)
    paged.K, paged.V, paged.table, paged.page = block.cache.k.cpu(), block.cache.v.cpu(), block.cache.table.cpu(), block.cache.page_size
    case = (torch.bfloat16, torch.float32, 4, 2, 64, [60] * 3, [1] * 3)
    check_attention(case, paged, qr.cpu(), None, out, lse, 64 ** -0.5)
