"""The cache calls from their definitions, in 64 bits, row by row (numpy), and
the paged caches the tests run them on.  Shares no code with the library."""
from __future__ import annotations

import numpy as np
import torch

U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}   # half an ulp of 1, as a ratio
E32 = 2.0 ** -24


class Paged:
    """B sequences with room for `slots` slots each, in shuffled pages; table
    None: one page per sequence.  Unused memory holds NaN."""

    def __init__(self, rng, B, slots, page, kv, dim, dtype, order="token", table=True, spare=2, pad=0):
        self.B, self.page, self.kv, self.dim, self.dtype = B, page, kv, dim, dtype
        per = -(-slots // page) if table else 1
        self.page = page = page if table else slots
        pages = B * per + (spare if table else 0)
        shape = (pages, page, kv, dim + pad) if order == "token" else (pages, kv, page, dim + pad)
        self.K, self.V = (torch.full(shape, float("nan"), dtype=dtype) for _ in range(2))
        if order == "head":
            self.K, self.V = self.K.transpose(1, 2), self.V.transpose(1, 2)
        self.K, self.V = self.K[..., :dim], self.V[..., :dim]
        self.table = torch.from_numpy(rng.permutation(pages)[: B * per].reshape(B, per).astype(np.int32)) if table else None
        self.slots = per * page

    def at(self, b, s):
        s = np.asarray(s)
        pages = self.table[b].numpy()[s // self.page] if self.table is not None else np.full(s.shape, b)
        return torch.from_numpy(np.asarray(pages, dtype=np.int64)), torch.from_numpy(np.asarray(s % self.page, dtype=np.int64))

    def get(self, which, b, s):
        p, o = self.at(b, s)
        return (self.K if which == "K" else self.V)[p, o].double().numpy()      # [n, kv, dim]

    def put(self, which, b, s, x):
        p, o = self.at(b, s)
        (self.K if which == "K" else self.V)[p, o] = torch.as_tensor(x).to(self.dtype)

    def device(self, bnn, pos=None, score=None):
        """The cache on the GPU, with the strides it has here."""
        def move(x):
            base = x
            out = torch.empty_strided(base.shape, base.stride(), dtype=base.dtype, device="cuda")
            out.copy_(base)
            return out
        self.dK, self.dV = move(self.K), move(self.V)
        self.dtable = None if self.table is None else self.table.cuda()
        return bnn.KVCache(self.dK, self.dV, self.dtable, pos=pos, score=score)


def sees(ctx, T, i, mask_row):
    """Which of the ctx + T slots new token i sees."""
    v = np.ones(ctx + T, dtype=bool)
    v[ctx:] = (np.arange(T) <= i) if mask_row is None else mask_row[:T]
    return v


def attention(q, k, v, vis, scale):
    """q [H, D], k, v [n, kv, D] float64, vis [n]: out [H, D], lse [H], and for
    the bounds A = sum p |v| [H, D], the largest scale sum |q k| [H] over seen slots."""
    H, D = q.shape
    g = H // k.shape[1]
    out, lse, A, S = np.zeros((H, D)), np.full(H, -np.inf), np.zeros((H, D)), np.zeros(H)
    kk, vv = k[vis], v[vis]
    if kk.shape[0] == 0:
        return out, lse, A, S
    for h in range(H):
        s = kk[:, h // g] @ q[h] * scale
        m = s.max()
        p = np.exp(s - m)
        t = p.sum()
        lse[h] = m + np.log(t)
        out[h] = (p / t) @ vv[:, h // g]
        A[h] = (p / t) @ np.abs(vv[:, h // g])
        S[h] = (np.abs(kk[:, h // g]) @ np.abs(q[h])).max() * scale
    return out, lse, A, S


def rope(x, w, eps, cos, sin, rot, interleaved):
    """x [n, H, D] float64; cos, sin [n, rot/2].  Returns y and |a c| + |b s| per element."""
    y = x.copy()
    if w is not None:
        y = y / np.sqrt((y * y).mean(-1, keepdims=True) + eps) * w
    half = rot // 2
    i = np.arange(half)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    c, s = cos[:, None], sin[:, None]
    z, mag = y.copy(), np.abs(y)
    z[..., a] = y[..., a] * c - y[..., b] * s
    z[..., b] = y[..., b] * c + y[..., a] * s
    mag[..., a] = np.abs(y[..., a] * c) + np.abs(y[..., b] * s)
    mag[..., b] = np.abs(y[..., b] * c) + np.abs(y[..., a] * s)
    return z, mag


def evict(ctx, T, accepted, budget, recent, pos, score):
    """One (sequence, head): pos, score [>= ctx + T].  Returns keep, the
    source slot of each of the first keep slots."""
    valid = [s for s in range(ctx)] + [ctx + i for i in range(T) if accepted is None or accepted[i]]
    keep = min(len(valid), budget)
    last = max((int(pos[s]) for s in valid), default=0)
    def rank(s):
        w = float(score[s])
        w = -np.inf if np.isnan(w) else w
        return (0 if int(pos[s]) > last - recent else 1, -w, s)
    def key(s):
        r = rank(s)
        return (0, 0.0, s) if r[0] == 0 else r
    stay = sorted(sorted(valid, key=key)[:keep])
    source = list(range(keep))
    for hole, mover in zip([s for s in range(keep) if s not in set(stay)], [s for s in stay if s >= keep]):
        source[hole] = mover
    return keep, np.array(source, dtype=np.int64)


def packed(rows, words):
    x = np.zeros((len(rows), words * 32), dtype=np.uint8)
    for r, on in enumerate(rows):
        x[r, list(on)] = 1
    return torch.from_numpy(np.packbits(x, axis=1, bitorder="little").view(np.int32).copy())


def random_tree(rng, T):
    """Parents of T nodes and the set each node sees (itself and ancestors)."""
    par = [int(rng.integers(-1, i)) if i else -1 for i in range(T)]
    seen = []
    for i, p in enumerate(par):
        seen.append((set(seen[p]) if p >= 0 else set()) | {i})
    return par, seen
