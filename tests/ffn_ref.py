"""The feed-forward calls from their definitions, in 64 bits (numpy), and what
their outputs may be off.  Shares no code with the library.

Half a step of a type, relative to the value: U.  An fp32 quotient, product or
sum is off by at most E32 of its value."""
from __future__ import annotations

import math

import numpy as np
import torch

U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
E32 = 2.0 ** -24
TINY = {torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -24, torch.float32: 2.0 ** -149}   # the smallest positive value


def rounded(x, dtype):
    """64-bit values through fp32 to `dtype`, as 64-bit values."""
    return torch.from_numpy(np.asarray(x, dtype=np.float64)).float().to(dtype).double().numpy()


def f64(t):
    return t.double().cpu().numpy()


# ---- block_norm


def norm(v, kind, w, b, eps):
    if kind == "none":
        return v
    with np.errstate(all="ignore"):
        if kind == "layer":
            v = v - v.mean(-1, keepdims=True)
        v = v / np.sqrt((v * v).mean(-1, keepdims=True) + float(np.float32(eps)))
        v = v if w is None else v * f64(w)
        return v if b is None else v + f64(b)


def quantized(y, by_quotient=False):
    """Codes, row scales and row sums of fp32 rows: single precision, one rounding a step, NaN skipped.
    ``by_quotient``: with 127 / amax as bnn_quantize_act_i8 has it, not 127 times the reciprocal."""
    y = y.astype(np.float32)
    with np.errstate(all="ignore"):
        a = np.abs(y)
        most = np.where(np.isnan(a), np.float32(0), a).max(-1, keepdims=True)
        inv = np.float32(127) / most if by_quotient else np.float32(1) / most * np.float32(127)
        inv = np.where(most > 0, inv, np.float32(0)).astype(np.float32)
        q = np.rint((y * inv).astype(np.float32))
        q = np.where(np.isnan(q), 0, np.clip(q, -127, 127)).astype(np.int8)
        return q, (most / np.float32(127)).astype(np.float32)[:, 0], q.astype(np.int32).sum(-1)


def planes(q, ld):
    """Bit planes [M, 8, ld] of codes."""
    M, K = q.shape
    u = q.view(np.uint8)
    bits = np.zeros((M, 8, ld * 32), dtype=np.uint8)
    for b in range(8):
        bits[:, b, :K] = (u >> b) & 1
    return np.packbits(bits, axis=-1, bitorder="little").view(np.int32)


def block_norm(x, branch, *, place=None, weight=None, post="none", post_weight=None, post_bias=None, gate=None, x_scale=1.0, branch_scale=1.0,
               pre="rms", pre_weight=None, pre_bias=None, eps=1e-6, store=True):
    """(stream before it is rounded, stream as it is stored, y in 64 bits)."""
    s = 0.0
    with np.errstate(all="ignore"):
        if branch is not None:
            b = f64(branch)
            if place is not None:
                p = place.cpu().numpy()
                w = np.ones(p.shape) if weight is None else f64(weight)
                rows = np.zeros((p.shape[0], b.shape[1]))
                for m in range(p.shape[0]):
                    for j in range(p.shape[1]):
                        if 0 <= p[m, j] < b.shape[0]:
                            rows[m] += w[m, j] * b[p[m, j]]
                b = rows
            b = norm(b, post, post_weight, post_bias, eps)
            b = b if gate is None else b * f64(gate)
            s = b * float(np.float32(branch_scale))
        if x is not None:
            s = s + float(np.float32(x_scale)) * f64(x)
        stored = rounded(s, x.dtype) if x is not None and store else s
        return s, stored, norm(stored, pre, pre_weight, pre_bias, eps)


# ---- expert_route


def expert_route(logits, top, *, score="softmax", bias=None, renorm=False, scale=1.0, used=None):
    """expert, weight (64 bits), offsets, order (only the taken entries), place; -9 in rows that are left alone."""
    l = f64(logits)
    rows, E = l.shape
    n = rows if used is None else max(0, min(rows, used))
    expert, place, weight = np.full((rows, top), -9), np.full((rows, top), -9), np.full((rows, top), -9.0)
    for r in range(n):
        x = np.where(np.isnan(l[r]), -np.inf, l[r])
        with np.errstate(all="ignore"):
            if score == "sigmoid":
                s = 1 / (1 + np.exp(-x))
            else:
                m = x.max()
                e = np.exp(x - (0.0 if m == -np.inf else m))
                s = e / e.sum() if e.sum() != 0 else e
        key = x if bias is None else np.where(x > -np.inf, s + f64(bias), -np.inf)
        key = np.where(np.isnan(key), -np.inf, key)
        by = sorted((i for i in range(E) if key[i] > -np.inf), key=lambda i: (-key[i], i))[:top]
        w = np.array([s[i] for i in by])
        if renorm and len(by):
            w = w / w.sum() if w.sum() != 0 else 0 * w
        expert[r], weight[r], place[r] = -1, 0.0, -1
        expert[r, :len(by)], weight[r, :len(by)] = by, w * float(np.float32(scale))
    order, offsets = [], [0]
    for e in range(E):
        pairs = np.flatnonzero((expert == e).reshape(-1))
        place.reshape(-1)[pairs] = len(order) + np.arange(len(pairs))
        order += pairs.tolist()
        offsets.append(len(order))
    return expert, weight, np.array(offsets), np.array(order, dtype=np.int64), place


# ---- expert_linear


def activated(z, act):
    with np.errstate(all="ignore"):
        if act == "relu":
            return np.where(z < 0, 0, z)
        if act == "relu2":
            return np.where(z < 0, 0, z) ** 2
        if act == "silu":
            return z / (1 + np.exp(-z))
        if act == "gelu":
            return z * 0.5 * np.vectorize(math.erfc, otypes=[np.float64])(-z / math.sqrt(2.0))
        if act == "gelu_tanh":
            return z * 0.5 * (1 + np.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
        return z


def slope(z, act):
    """A bound of |act'| near z, and what the activation's own evaluation is off, absolutely, besides a rounding of z:
    expf and erfcf are within 2 ulp; expf(-z) of a rounded argument is off by |z| E32 relative, erfcf(u) by about 2 u^2 2^-24."""
    a = np.abs(activated(z, act))
    if act == "relu2":
        return 2 * np.abs(z) + 1e-30, 2 * E32 * a
    if act in ("silu", "gelu_tanh"):
        t = np.abs(z) if act == "silu" else np.abs(1.5957691216 * (z + 0.044715 * z ** 3))
        return 1.2 + 0 * z, (8 + 6 * t) * E32 * a     # the argument's own roundings (up to 5 of them), the exponential's, sum, quotient
    if act == "gelu":
        return 1.2 + 0 * z, (16 + 4 * z * z) * E32 * a
    return 1.0 + 0 * z, 0 * a


def expert_linear(Xq, t, alpha, *, xscale=None, bias=None, order=None, per_row=1, offsets=None, act="none", up=None, residual=None):
    """(y in 64 bits, a bound of its fp32 error, the positions that are written).  t: [E, N, K] whole numbers; up: (t, alpha, bias)."""
    q, E = Xq.cpu().numpy().astype(np.int64), t.shape[0]
    P = len(order) if order is not None else q.shape[0]
    ends = [0, P] if offsets is None else np.asarray(offsets).tolist()
    N = t.shape[1]
    y, off, live = np.zeros((P, N)), np.zeros((P, N)), np.zeros(P, dtype=bool)
    for e in range(E):
        at = np.arange(ends[e], ends[e + 1])
        rows = np.asarray(order)[at] // per_row if order is not None else at
        ok = (rows >= 0) & (rows < q.shape[0])
        at, rows = at[ok], rows[ok]
        live[at] = True
        xs = np.ones(len(at)) if xscale is None else f64(xscale)[rows]

        def product(t, alpha, bias):
            a = f64(alpha)
            z = (q[rows] @ t[e].astype(np.int64).T) * (a[e] if a.ndim == 1 else a[e][None]) * xs[:, None]
            err = 2 * E32 * np.abs(z) * 1.01      # alpha D, times xscale
            if bias is not None:
                z = z + f64(bias)[e]
                err = err + E32 * np.abs(z) * 1.01
            return z, err

        z, err = product(t, alpha, bias)
        s, own = slope(z, act)
        v, verr = activated(z, act), err * s * 1.01 + own
        if act == "relu2":
            verr = verr + err * err
        if up is not None:
            u, uerr = product(*up)
            verr = verr * np.abs(u) + np.abs(v) * uerr + verr * uerr
            v = v * u
            verr = verr + E32 * np.abs(v) * 1.01
        if residual is not None:
            v = v + f64(residual)[at]
            verr = verr + E32 * np.abs(v) * 1.01
        y[at], off[at] = v, verr
    return y, off, live
