"""GPU checks of the calls over the paged key/value cache at the edges of their
definitions: weights far below one that dominates its row, evictions where the
recent tokens alone exceed the budget, workspaces made for other sizes, steps without
new tokens, infinities and NaN among the committed tokens,
pages that are not there, launches of more than 2^24 workgroups, trees of more
nodes than a word has bits.

Bounds as in test_gpu_cache.py: u is half an ulp of a type as a ratio, products
and sums in fp32 add (D + 10) 2^-24 sum |q k| scale to a logit and n 2^-24 to a
sum."""
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


# ---- weights far below the row's largest

@pytest.mark.parametrize("gap", [10.0, 12.0, 14.0, 16.0, 18.0])
@pytest.mark.parametrize("out", [FP, torch.float32], ids=["f16", "f32"])
@pytest.mark.parametrize("T", [1, 8, 16, 24])     # 4, 32, 64, 96 rows of a key head: each kernel
def test_attention_one_token_dominates(bnn, T, out, gap):
    """float16: the first slot's logit is `gap` above all others and its V is 0,
    so the output is made of the small weights alone.  32 sequences share the
    pages, so that a chunk holds thousands of slots."""
    banner(f"tree_attention dominated T={T} {out} gap={gap}")
    rng = np.random.default_rng(41)
    B, heads, kv, dim, n, page, u = 32, 64, 16, 64, 4000, 64, ref.U[FP]
    cache = ref.Paged(rng, 1, n + T, page, kv, dim, FP)
    direction = np.sign(rng.standard_normal(dim))
    scale = dim ** -0.5
    k, v = rng.standard_normal((2, n + T, kv, dim)) * np.array([0.3, 1.0])[:, None, None, None]
    k -= (k @ direction / dim)[..., None] * direction          # nothing along the direction ...
    k[0] = direction * (gap / (dim * scale))                   # ... but the first slot's
    v[0] = 0
    cache.put("K", 0, np.arange(n + T), k)
    cache.put("V", 0, np.arange(n + T), v)
    q = torch.from_numpy(direction + 0.05 * rng.standard_normal((T, heads, dim))).to(FP)
    mask = bnn.tree_mask([-1] * T)                             # every token sees itself of the new ones
    one = cache.device(bnn)
    dc = bnn.KVCache(one.k, one.v, one.table.expand(B, -1).contiguous())
    got, lse = bnn.tree_attention(q.cuda().repeat(B, 1, 1), dc, cuda_i32([T * b for b in range(B + 1)]), cuda_i32([n] * B), max_nodes=T, max_ctx=n,
                                  mask=mask.cuda().repeat(B, 1), scale=scale, out_dtype=out)
    torch.cuda.synchronize()
    got, lse = got.double().cpu().numpy().reshape(B, T, heads, dim), lse.double().cpu().numpy().reshape(B, T, heads)
    assert (got == got[:1]).all() and (lse == lse[:1]).all()
    k, v = (cache.get(w, 0, np.arange(n + T)) for w in "KV")
    blocks = [slice(s, min(s + 64, n + T)) for s in range(0, n + T, 64)]
    for i in range(T):
        vis = ref.sees(n, T, i, np.arange(T) == i)
        y, l, A, S = ref.attention(q[i].double().numpy(), k, v, vis, scale)
        ds = (dim + 10) * ref.E32 * S
        assert (np.abs(lse[0, i] - l) <= ds + (n + 8) * ref.E32 + 8 * ref.E32 * np.abs(l)).all()
        for h in range(heads):
            w = np.where(vis, np.exp(k[:, h // 4] @ q[i, h].double().numpy() * scale - l[h]), 0)
            far = sum(w[s].max() * np.abs(v[s, h // 4]).sum(0) for s in blocks) * 2.0 ** -30
            own = 2.0 ** -22 * A[h] + ref.E32 * np.abs(y[h]) if out == torch.float32 else u * (A[h] + np.abs(y[h])) + 2.0 ** -25
            # a matrix product adds 16 or 32 slots and rounds the sum once, so a chain is n / 16 long
            bound = own + far + (2 * ds[h] + 2 * (n / 16 + 40) * ref.E32) * A[h]
            err = np.abs(got[0, i, h] - y[h])
            assert (err <= bound).all(), (i, h, float((err / bound).max()), float((err / np.abs(y[h])).max()))


# ---- recent tokens that alone exceed the budget

def evict_by_rank(ctx, accepted, budget, recent, pos, score):
    """One (sequence, head) by the definition: recent tokens first, then by
    score (NaN as -inf), equal scores by slot.  Returns the source slot of each
    kept one."""
    valid = np.concatenate((np.arange(ctx), ctx + np.flatnonzero(accepted))).astype(np.int64)
    keep = min(len(valid), budget)
    w = np.where(np.isnan(score[valid]), -np.inf, score[valid].astype(np.float64))
    late = pos[valid].astype(np.int64) > (int(pos[valid].max()) - recent if len(valid) else 0)
    stay = np.sort(valid[np.lexsort((valid, -w, ~late))[:keep]])
    source = np.arange(keep)
    source[np.setdiff1d(source, stay)] = stay[stay >= keep]
    return source


@pytest.mark.parametrize("inplace", (False, True))
@pytest.mark.parametrize("case", [
    # ctx, nodes, budget, recent
    ([12], [1], 4, 100), ([1500], [3], 700, 2000), ([0, 1, 90, 300], [9, 3, 0, 5], 7, 40), ([3000], [8], 64, 64), ([3000], [8], 64, 65),
    ([3000], [8], 64, 63), ([7000, 60], [31, 31], 1, 1 << 40), ([14000], [2], 5000, 9000), ([30000], [1], 300, 20000),
    ([40000, 33000], [1, 64], 2500, 30000), ([500], [4], 0, 300)], ids=range(11))
def test_evict_more_recent_tokens_than_the_budget(bnn, case, inplace):
    ctx, nodes, budget, recent = case
    banner(f"cache_evict recent over the budget {case} inplace={inplace}")
    rng = np.random.default_rng(51)
    B, kv, dim = len(ctx), 2, 64
    cache = ref.Paged(rng, B, max(c + t for c, t in zip(ctx, nodes)) + 2, 16, kv, dim, BF)
    pos = np.full((B, kv, cache.slots), -3, dtype=np.int32)
    score = np.full((B, kv, cache.slots), 2.5, dtype=np.float32)
    accepted = [rng.random(t) < 0.6 for t in nodes]
    for b in range(B):
        n = ctx[b] + nodes[b]
        for w in "KV":
            cache.put(w, b, np.arange(n), rng.standard_normal((n, kv, dim)))
        for h in range(kv):
            pos[b, h, :n] = rng.permutation(n)
            x = rng.standard_normal(n).astype(np.float32) ** 2
            x[rng.random(n) < 0.3] = rng.choice(np.array([0.0, -0.0, 1.0, np.inf, -np.inf, np.nan], dtype=np.float32))
            score[b, h, :n] = x
    before = cache.K.clone(), cache.V.clone()
    dpos, dscore, dctx = torch.from_numpy(pos.copy()).cuda(), torch.from_numpy(score.copy()).cuda(), cuda_i32(ctx)
    dc = cache.device(bnn, dpos, dscore)
    kw = {} if inplace else dict(pos_out=torch.full_like(dpos, -9), score_out=torch.full_like(dscore, -9.0), ctx_out=torch.full_like(dctx, -9))
    got = bnn.cache_evict(dc, cuda_i32(np.concatenate(([0], np.cumsum(nodes)))), dctx, budget=budget, recent=recent, max_nodes=max(nodes),
                          max_ctx=max(ctx), accept=ref.packed([np.flatnonzero(a) for a in accepted], 2).cuda(), **kw)
    torch.cuda.synchronize()
    pos2, score2 = (x.cpu().numpy() for x in ((dpos, dscore) if inplace else (kw["pos_out"], kw["score_out"])))
    wantK, wantV = before[0].clone(), before[1].clone()
    for b in range(B):
        n = ctx[b] + nodes[b]
        for h in range(kv):
            source = evict_by_rank(ctx[b], accepted[b], budget, recent, pos[b, h, :n], score[b, h, :n])
            keep = len(source)
            assert got[b] == keep
            assert np.array_equal(pos2[b, h, :keep], pos[b, h, source]) and (pos2[b, h, keep:n] == -1).all()
            assert np.array_equal(score2[b, h, :keep].view(np.int32), score[b, h, source].view(np.int32)) and (score2[b, h, keep:n] == 0).all()
            if keep:
                to, come = cache.at(b, np.arange(keep)), cache.at(b, source)
                wantK[(*to, h)], wantV[(*to, h)] = before[0][(*come, h)], before[1][(*come, h)]
    same = lambda x, y: torch.equal(x.contiguous().view(torch.int16), y.contiguous().view(torch.int16))
    assert same(cache.dK.cpu(), wantK) and same(cache.dV.cpu(), wantV)


# ---- workspaces

@pytest.mark.parametrize("heads,kv,dim,seqs,nodes,ctx", [(8, 2, 128, 64, 1, 1500), (8, 2, 64, 5, 70, 3000), (4, 4, 256, 3, 9, 2500)])
def test_attention_with_a_workspace_of_other_sizes(bnn, heads, kv, dim, seqs, nodes, ctx):
    """A workspace for more sequences and tokens, one that holds two chunks,
    and none at all: the same function."""
    banner(f"tree_attention workspaces {heads} {kv} {dim} {seqs} {nodes} {ctx}")
    gen = torch.Generator(device="cuda").manual_seed(61)
    normal = lambda *shape: torch.randn(shape, generator=gen, device="cuda").to(BF)
    per = -(-(ctx + nodes) // 64)
    table = torch.arange(seqs * per, dtype=torch.int32, device="cuda").reshape(seqs, per)
    cache = bnn.KVCache(normal(seqs * per, 64, kv, dim), normal(seqs * per, 64, kv, dim), table)
    work = bnn.tree_attention_workspace(cache, seqs * nodes, heads, nodes, ctx)
    for b, n, spare in ((1, 1, 0), (1, nodes, 0), (seqs, 1, 3), (2, nodes, 300)):
        rows = b * n
        q = normal(rows + spare, heads, dim)
        args = dict(max_nodes=n, max_ctx=ctx, out_dtype=torch.float32)
        indptr, held = cuda_i32(range(0, rows + 1, n)), cuda_i32([ctx - 7 * i for i in range(b)])
        two = torch.empty(2 * q.shape[0] * heads * (4 * dim + 8), dtype=torch.uint8, device="cuda")
        results = [bnn.tree_attention(q, cache, indptr, held, workspace=w, **args) for w in (None, work, two, two[:0], two[:4096])]
        # one row by its definition, the others alike.  A logit's products are off by (D + 10) 2^-24 scale sum |q k|, at most
        # 266 x 6e-8 x 12 = 2e-4 here (normal values), a weight by as much again for lse, and the mean of |v| is 0.8
        k, v = (x[table[0].long()].flatten(0, 1)[: ctx + 1].double() for x in (cache.k, cache.v))
        for h in range(heads):
            s = (k[:, h * kv // heads] @ q[0, h].double()) * dim ** -0.5
            want = torch.softmax(s, 0) @ v[:, h * kv // heads]
            for out, lse in results:
                assert torch.allclose(out[0, h].double(), want, rtol=0, atol=4e-4) and abs(float(lse[0, h]) - float(torch.logsumexp(s, 0))) < 2e-4
        for out, lse in results[1:]:
            assert torch.allclose(out[:rows], results[0][0][:rows], rtol=0, atol=8e-4) and torch.allclose(lse[:rows], results[0][1][:rows], rtol=0, atol=4e-4)


# ---- nothing to do

def no_tokens(B, kv=2, heads=4, dim=64, n=40):
    gen = torch.Generator(device="cuda").manual_seed(71)
    normal = lambda *shape: torch.randn(shape, generator=gen, device="cuda")
    per = -(-n // 16)
    K, V = normal(B * per + 1, 16, kv, dim).to(BF), normal(B * per + 1, 16, kv, dim).to(BF)
    pos = torch.stack([torch.randperm(per * 16, generator=gen, device="cuda") for _ in range(B * kv)]) if B else torch.empty(0, device="cuda")
    return (K, V, torch.arange(B * per, dtype=torch.int32, device="cuda").reshape(B, per), pos.to(torch.int32).reshape(B, kv, per * 16).contiguous(),
            normal(B, kv, per * 16).abs())


@pytest.mark.parametrize("B", [0, 3])
def test_a_step_without_new_tokens(bnn, B):
    """No rows (every sequence waits), and no sequences: the calls do what is
    left to do, which for the sums is the copy and for the eviction the cut."""
    banner(f"no rows, {B} sequences")
    K, V, table, pos, score = no_tokens(B)
    kept = [x.clone() for x in (K, V, pos, score)]
    cache = bnn.KVCache(K, V, table, pos=pos, score=score)
    indptr, ctx = cuda_i32([0] * (B + 1)), cuda_i32([40] * B)
    q, k = torch.empty((0, 4, 64), device="cuda"), torch.empty((0, 2, 64), device="cuda")
    qr = bnn.qk_norm_rope(q, k, k, cache, indptr, ctx, cuda_i32([]), bnn.rope_turns(50, 64, device="cuda"))
    assert qr.shape == (0, 4, 64) and qr.dtype == BF
    mask, accept = torch.empty((0, 1), dtype=torch.int32, device="cuda"), torch.zeros((B, 1), dtype=torch.int32, device="cuda")
    args = dict(max_nodes=5, max_ctx=40)
    out, lse = bnn.tree_attention(qr, cache, indptr, ctx, mask=mask, **args)
    assert out.shape == (0, 4, 64) and lse.shape == (0, 4)
    res = torch.full_like(score, 9.0)
    assert bnn.cache_score_add(qr, lse, cache, indptr, ctx, mask=mask, accept=accept, score_out=res, **args) is res and torch.equal(res, score)
    bnn.cache_score_add(qr, lse, cache, indptr, ctx, **args)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip((K, V, pos, score), kept))
    got = bnn.cache_evict(cache, indptr, ctx, budget=25, recent=0, accept=accept, **args)
    assert got.tolist() == [25] * B
    for b in range(B):
        for h in range(2):
            source = evict_by_rank(40, np.zeros(0, dtype=bool), 25, 0, kept[2][b, h].cpu().numpy(), kept[3][b, h].cpu().numpy())
            assert np.array_equal(pos[b, h, :25].cpu().numpy(), kept[2][b, h].cpu().numpy()[source]) and (pos[b, h, 25:40] == -1).all()


def test_no_pages_and_no_table_of_angles(bnn):
    """A cache without pages holds nothing; a table without positions gives NaN."""
    banner("no pages")
    K = torch.empty((0, 16, 2, 64), dtype=BF, device="cuda")
    cache = bnn.KVCache(K, K.clone(), torch.zeros((2, 3), dtype=torch.int32, device="cuda"))
    q, k = torch.randn((2, 4, 64), device="cuda"), torch.randn((2, 2, 64), device="cuda")
    indptr, ctx = cuda_i32([0, 1, 2]), cuda_i32([0, 5])
    qr = bnn.qk_norm_rope(q, k, k, cache, indptr, ctx, cuda_i32([0, 1]), bnn.rope_turns(0, 32, device="cuda"))
    assert qr[..., :32].isnan().all() and torch.equal(qr[..., 32:], q[..., 32:].to(BF))
    out, lse = bnn.tree_attention(q.to(BF), cache, indptr, ctx, max_nodes=1, max_ctx=5)
    # missing pages read as rows of zeros: logits 0, values 0
    assert (out == 0).all() and torch.allclose(lse, torch.tensor([[0.0] * 4, [6.0] * 4], device="cuda").clamp(min=1).log(), rtol=0, atol=1e-6)


# ---- infinities among the committed tokens

@pytest.mark.parametrize("kind", [BF, FP], ids=["bf16", "f16"])
@pytest.mark.parametrize("T,heads,kv,dim", [(1, 4, 1, 128), (1, 2, 2, 64), (9, 8, 2, 96), (70, 16, 2, 64), (3, 8, 1, 256)])
def test_score_of_infinite_keys(bnn, T, heads, kv, dim, kind):
    """Committed keys that hold an infinity: a logit of -inf adds nothing, one
    of +inf adds infinity, NaN adds NaN; rows that are not there and rows that
    saw nothing add nothing to either."""
    banner(f"cache_score_add infinite keys T={T} {kind}")
    rng = np.random.default_rng(81)
    n, g, scale = 150, heads // kv, dim ** -0.5
    cache = ref.Paged(rng, 1, n + T, 16, kv, dim, kind)
    k = rng.standard_normal((n + T, kv, dim))
    k[40, :, 3], k[41, :, 3], k[70, :, 3], k[71, 0, 5] = -np.inf, np.inf, -np.inf, np.nan
    cache.put("K", 0, np.arange(n + T), k)
    cache.put("V", 0, np.arange(n + T), np.zeros((n + T, kv, dim)))
    q = torch.from_numpy(rng.standard_normal((T, heads, dim)) * 0.5)
    q[..., 3] = q[..., 3].abs() + 0.25
    q = q.to(kind)
    lse = torch.from_numpy(rng.standard_normal((T, heads)) + 4).float()
    lse[0, 0] = float("-inf")
    score = torch.from_numpy(rng.random((1, kv, cache.slots))).float()
    dc = cache.device(bnn, score=score.cuda())
    got = bnn.cache_score_add(q.cuda(), lse.cuda(), dc, cuda_i32([0, T]), cuda_i32([n]), max_nodes=T, max_ctx=n, scale=scale).double().cpu().numpy()[0]
    k = cache.get("K", 0, np.arange(n + T))
    want, tol = score[0, :, : n + T].double().numpy().copy(), np.zeros((kv, n + T))
    with np.errstate(invalid="ignore"):
        for i in range(T):
            for h in range(heads):
                if not torch.isneginf(lse[i, h]):
                    x = k[: n + i + 1, h // g] @ q[i, h].double().numpy() * scale
                    S = np.abs(k[: n + i + 1, h // g]) @ np.abs(q[i, h].double().numpy()) * scale
                    w = np.exp(x - float(lse[i, h]))
                    want[h // g, : n + i + 1] += w
                    finite = np.isfinite(x)
                    tol[h // g, : n + i + 1][finite] += (w * ((dim + 10) * S + 8 * np.abs(x) + 8 * abs(float(lse[i, h])) + 8 + T * g) * ref.E32)[finite]
    assert np.isfinite(want[:, 40]).all()
    if T * g > 1:                               # else head 0 has the one row that saw nothing
        assert np.isnan(want[0, 71]) and np.isinf(want[:, 41]).all()
    got = got[:, : n + T]
    finite = np.isfinite(want)
    assert np.array_equal(got[~finite], want[~finite], equal_nan=True)
    assert (np.abs(got[finite] - want[finite]) <= (tol + 2 * ref.E32 * np.abs(want))[finite]).all()


# ---- NaN logits

@pytest.mark.parametrize("out", [BF, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("T,heads,kv,dim,ctx", [(1, 4, 1, 128, 60), (1, 4, 1, 128, 5000), (7, 8, 2, 64, 5000), (15, 8, 2, 96, 900), (40, 8, 2, 128, 5000),
                                                (40, 8, 2, 256, 3000)])
def test_attention_of_nan_rows(bnn, T, heads, kv, dim, ctx, out):
    """A query that holds NaN gives NaN in its row and head alone; NaN in the
    keys of a whole run of committed slots gives it to every row of that key
    head; however many chunks the slots are cut into."""
    banner(f"tree_attention NaN T={T} dim={dim} ctx={ctx} {out}")
    rng = np.random.default_rng(91)
    cache = ref.Paged(rng, 1, ctx + T, 16, kv, dim, BF)
    for w in "KV":
        cache.put(w, 0, np.arange(ctx + T), rng.standard_normal((ctx + T, kv, dim)))
    q = torch.from_numpy(rng.standard_normal((T, heads, dim))).to(BF)
    args = dict(max_nodes=T, max_ctx=ctx, out_dtype=out)
    run = lambda q: bnn.tree_attention(q.cuda(), cache.device(bnn), cuda_i32([0, T]), cuda_i32([ctx]), **args)
    whole, lse0 = run(q)
    assert not whole.isnan().any() and not lse0.isnan().any()
    bad = q.clone()
    bad[T // 2, 1, 5] = float("nan")
    got, lse = run(bad)
    assert got[T // 2, 1].isnan().all() and lse[T // 2, 1].isnan()
    rest = torch.ones(T, heads, dtype=torch.bool)
    rest[T // 2, 1] = False
    assert torch.equal(got.cpu()[rest], whole.cpu()[rest]) and torch.equal(lse.cpu()[rest], lse0.cpu()[rest])
    first = np.arange(min(ctx, 300))
    k = cache.get("K", 0, first)
    k[:, 0, 2] = np.nan
    cache.put("K", 0, first, k)
    got, lse = run(q)
    g = heads // kv
    assert got[:, :g].isnan().all() and lse[:, :g].isnan().all()
    assert torch.equal(got[:, g:], whole[:, g:]) and torch.equal(lse[:, g:], lse0[:, g:])


# ---- infinities among the committed values

@pytest.mark.parametrize("out", ["same", "f32"])
@pytest.mark.parametrize("kind", [BF, FP], ids=["bf16", "f16"])
@pytest.mark.parametrize("T,heads,kv,dim,ctx,page", [(1, 4, 2, 128, 40, 16), (1, 4, 2, 64, 3000, 16), (7, 8, 2, 96, 1500, 1), (15, 8, 2, 128, 700, 24),
                                                     (40, 8, 2, 128, 3000, 64), (200, 4, 2, 64, 300, 64), (20, 8, 2, 256, 900, 16), (2, 8, 2, 256, 2000, 16)])
def test_attention_of_infinite_values(bnn, T, heads, kv, dim, ctx, page, kind, out):
    """Values that hold infinities of one sign, of both, and NaN give
    infinity or NaN in that dimension to every row, however small their weight
    (the last of them lie 100 below the largest logit); other dimensions are
    as the definition says."""
    banner(f"tree_attention infinite values T={T} dim={dim} ctx={ctx} {kind} {out}")
    rng = np.random.default_rng(101)
    n, scale = ctx + T, dim ** -0.5
    out = kind if out == "same" else torch.float32
    cache = ref.Paged(rng, 1, n, page, kv, dim, kind)
    direction = np.sign(rng.standard_normal(dim))
    k, v = rng.standard_normal((2, n, kv, dim)) * np.array([0.5, 1.0])[:, None, None, None]
    far = ctx - 3
    k[far] = -direction * (100 / (dim * scale))
    inf = np.inf
    v[5, :, 7], v[ctx // 2, :, 11], v[ctx // 3, :, 12], v[ctx // 3 + 1, :, 12], v[9, :, 13] = inf, -inf, inf, -inf, np.nan
    v[far, :, 14], v[far, :, dim - 1], v[far - 1, 0, 20] = inf, -inf, inf
    v[ctx + T // 2, 1, 22], v[ctx, 0, 23], v[ctx + T - 1, :, 24] = -inf, inf, np.nan    # new tokens that some rows see
    for w, x in (("K", k), ("V", v)):
        cache.put(w, 0, np.arange(n), x)
    q = torch.from_numpy(direction + 0.3 * rng.standard_normal((T, heads, dim))).to(kind)
    got, lse = bnn.tree_attention(q.cuda(), cache.device(bnn), cuda_i32([0, T]), cuda_i32([ctx]), max_nodes=T, max_ctx=ctx, scale=scale, out_dtype=out)
    torch.cuda.synchronize()
    got, lse = got.double().cpu().numpy(), lse.double().cpu().numpy()
    k, v = (cache.get(w, 0, np.arange(n)) for w in "KV")
    u = ref.U[out] + (ref.U[kind] if out == kind else 2.0 ** -22) + 2.0 ** -24
    for i in range(T):
        with np.errstate(invalid="ignore"):
            y, l, A, S = ref.attention(q[i].double().numpy(), k, v, ref.sees(ctx, T, i, None), scale)
        assert np.isposinf(y[:, [7, 14]]).all() and np.isneginf(y[:, [11, dim - 1]]).all() and np.isnan(y[:, 12:14]).all() and np.isposinf(y[0, 20])
        odd = ~np.isfinite(y)
        assert np.array_equal(got[i][odd], y[odd], equal_nan=True), i
        ds = (dim + 10) * ref.E32 * S
        assert (np.abs(lse[i] - l) <= ds + (n + 8) * ref.E32 + 8 * ref.E32 * np.abs(l)).all()
        bound = u * np.where(odd, 0, A) + (2 * ds + 2 * n * ref.E32)[:, None] * np.where(odd, 0, A) + 2.0 ** -24
        assert (np.abs(got[i][~odd] - y[~odd]) <= bound[~odd]).all(), i


# ---- pages that are not there

@pytest.mark.parametrize("bad", [-1, 1 << 30])
def test_evict_missing_pages(bnn, bad):
    """A kept token whose page is not there reads as zeros, also once it has
    moved; one that moves to a page that is not there is not written."""
    banner(f"cache_evict missing page {bad}")
    rng = np.random.default_rng(111)
    n, kv, dim, keep = 96, 2, 64, 40
    cache = ref.Paged(rng, 1, n, 16, kv, dim, BF)
    for w in "KV":
        cache.put(w, 0, np.arange(n), rng.standard_normal((n, kv, dim)))
    cache.table[0, [1, 4]] = bad                  # slots 16-31 and 64-79
    pos = np.stack([rng.permutation(n) for _ in range(kv)])[None].astype(np.int32)
    score = rng.random((1, kv, n)).astype(np.float32)
    dpos, dscore = torch.from_numpy(pos.copy()).cuda(), torch.from_numpy(score.copy()).cuda()
    K, V = cache.K.clone(), cache.V.clone()
    dc = cache.device(bnn, dpos, dscore)
    bnn.cache_evict(dc, cuda_i32([0, 0]), cuda_i32([n]), budget=keep, recent=0, max_nodes=0, max_ctx=n)
    torch.cuda.synchronize()
    there = lambda s: s // 16 not in (1, 4)
    moved_from_nowhere = 0
    for h in range(kv):
        source = evict_by_rank(n, np.zeros(0, dtype=bool), keep, 0, pos[0, h], score[0, h])
        assert np.array_equal(dpos.cpu().numpy()[0, h, :keep], pos[0, h, source]) and np.array_equal(dscore.cpu().numpy()[0, h, :keep], score[0, h, source])
        for to, come in enumerate(source):
            if to != come and there(to):
                moved_from_nowhere += not there(come)
                for x in (K, V):
                    page, at = cache.at(0, [to])
                    x[page, at, h] = x[(*cache.at(0, [come]), h)] if there(come) else 0
    assert moved_from_nowhere > 0
    same = lambda x, y: torch.equal(x.contiguous().view(torch.int16), y.contiguous().view(torch.int16))
    assert same(dc.k.cpu(), K) and same(dc.v.cpu(), V)


# ---- more workgroups than one dimension of a launch takes

def test_append_of_very_many_rows(bnn):
    """2^24 + 3 new tokens, of which the cache has room for 16."""
    banner("qk_norm_rope 2^24 + 3 rows")
    rows = (1 << 24) + 3
    q = torch.zeros((rows, 1, 64), dtype=BF, device="cuda")
    q[-1], q[1 << 20], q[(1 << 20) - 1] = 1.0, 2.0, 3.0
    k = torch.ones((1, 1, 64), dtype=BF, device="cuda").expand(rows, 1, 64)
    K = torch.zeros((2, 16, 1, 64), dtype=BF, device="cuda")
    cache = bnn.KVCache(K, torch.zeros_like(K))
    out = torch.full_like(q, 7.0)
    bnn.qk_norm_rope(q, k, k, cache, cuda_i32([0, rows - 1, rows]), cuda_i32([0, 5]), torch.zeros(rows, dtype=torch.int32, device="cuda"), None, q_out=out)
    assert torch.equal(out, q)
    want = torch.zeros_like(K)
    want[0], want[1, 5] = 1, 1
    assert torch.equal(K, want)


def test_attention_of_very_many_workgroups(bnn):
    """65535 sequences of 257 heads, one token each over one slot of a shared
    page: each output is the slot's value of its head."""
    banner("tree_attention 65535 x 257 workgroups")
    B, heads = 65535, 257
    K, V = torch.zeros((2, 2, heads, 64), dtype=BF, device="cuda"), torch.randn((2, 2, heads, 64), device="cuda").to(BF)
    cache = bnn.KVCache(K, V, (torch.arange(B, dtype=torch.int32, device="cuda") % 2)[:, None].contiguous())
    q = torch.zeros((1, heads, 64), dtype=BF, device="cuda").expand(B, heads, 64)
    out, lse = bnn.tree_attention(q, cache, torch.arange(B + 1, dtype=torch.int32, device="cuda"), torch.zeros(B, dtype=torch.int32, device="cuda"),
                                  max_nodes=1, max_ctx=0)
    assert torch.equal(out.view(torch.int16)[0::2], V[0, 0].view(torch.int16).expand(B - B // 2, -1, -1))
    assert torch.equal(out.view(torch.int16)[1::2], V[1, 0].view(torch.int16).expand(B // 2, -1, -1)) and (lse == 0).all()


def test_attention_join_of_very_many_rows(bnn):
    """A token buffer of 2^24 + 3 rows whose sequences are cut into chunks."""
    banner("tree_attention 2^24 + 3 rows, two chunks")
    rows = (1 << 24) + 3
    K, V = torch.zeros((2, 512, 1, 64), dtype=BF, device="cuda"), torch.randn((2, 512, 1, 64), device="cuda").to(BF)
    cache = bnn.KVCache(K, V)
    q = torch.zeros((1, 1, 64), dtype=BF, device="cuda").expand(rows, 1, 64)
    out = torch.full((rows, 1, 64), 7.0, dtype=torch.float32, device="cuda")
    work = torch.empty(2 * rows * (64 * 4 + 8), dtype=torch.uint8, device="cuda")
    lse = torch.full((rows, 1), 7.0, device="cuda")
    # all rows but two are the first sequence's; two tokens of each get an output
    bnn.tree_attention(q, cache, cuda_i32([0, rows - 2, rows]), cuda_i32([300, 300]), max_nodes=2, max_ctx=300, out=out, lse=lse, workspace=work)
    assert (out[2:-2] == 7).all() and (lse[2:-2] == 7).all()
    for i, b, n in ((0, 0, 301), (1, 0, 302), (rows - 2, 1, 301), (rows - 1, 1, 302)):
        # equal weights: the mean of n values of 8 bits, n roundings of a sum below 4 n, which is then divided by n
        assert torch.allclose(out[i, 0], V[b, :n, 0].double().mean(0).float(), rtol=0, atol=4 * n * 2.0 ** -24)
        assert abs(float(lse[i]) - np.log(n)) < 8 * 2.0 ** -24 * 6


# ---- trees of more nodes than a word has bits

def test_example_of_wide_trees(bnn):
    """The example's path with 70 drafts: while the budget lasts the cache holds
    every accepted token."""
    banner("examples/decode_tree.py, 70 nodes")
    import os
    import sys
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import decode_tree
    block, y, length = decode_tree.run(steps=8, sequences=3, hidden=256, heads=4, kv_heads=2, dim=64, budget=400, recent=16, nodes=70)
    torch.cuda.synchronize()
    assert y.isfinite().all() and max(length) < 400 and block.ctx.tolist() == length
    for b in range(3):
        for h in range(2):
            assert sorted(block.cache.pos[b, h, : length[b]].tolist()) == list(range(length[b]))
