"""GPU checks of the calls over the paged key/value cache at the edges of their
definitions: weights far below one that dominates its row.

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
