"""Plain 64-bit forms of the operators around the attention step (expert routing, grouped 4-bit products, adapters,
log probabilities) with the bounds of their kernels' roundings, shared by their tests.  Nothing here uses the library."""
from __future__ import annotations

import numpy as np

H32 = 2.0 ** -24   # half a step of fp32, bf16 and of a tensor-core accumulation (which may cut off)
HBF = 2.0 ** -8
ACC = 2.0 ** -22


def route(logits, k, bias=None, active=None, renorm=True, scale=1.0):
    """(experts, weights, offsets, src, pos); logits float32 [m, E]."""
    m, E = logits.shape
    key = (logits + bias).astype(np.float32) if bias is not None else logits
    key = np.where(np.isnan(key), -np.inf, key).astype(np.float64)
    on = np.ones(m, bool) if active is None else np.asarray(active) != 0
    experts = np.full((m, k), -1, np.int64)
    weights = np.zeros((m, k))
    lists = [[] for _ in range(E)]
    for t in range(m):
        if not on[t]:
            continue
        order = sorted(range(E), key=lambda e: (-key[t, e], e))[:k]
        l = np.where(np.isnan(logits[t]), -np.inf, logits[t]).astype(np.float64)
        among = l[order] if renorm else l
        top = among.max()
        if top > -np.inf:
            p = lambda v: np.where(v == top, 1.0, np.exp(np.where(v == top, 0, v - top)))  # noqa: E731
            weights[t] = scale * p(l[order]) / p(among).sum()
        experts[t] = order
        for j, e in enumerate(order):
            lists[e].append((t, j))
    offsets = np.concatenate(([0], np.cumsum([len(v) for v in lists])))
    src, pos = np.full(m * k, -1, np.int64), np.full((m, k), -1, np.int64)
    for e in range(E):
        for i, (t, j) in enumerate(lists[e]):
            src[offsets[e] + i], pos[t, j] = t, offsets[e] + i
    return experts, weights, offsets, src, pos


def route_tol(logits, weights):
    """exp's argument (a difference of fp32 values, 2^-24 of it), exp itself (2 ulp), up to 37 additions, the division
    and the product with scale."""
    f = np.where(np.isfinite(logits), logits, 0.0)
    span = f.max(-1) - f.min(-1) if f.size else np.zeros(f.shape[0])
    return np.abs(weights) * (2 * span[:, None] + 64) * H32 * 2 + 2.0 ** -140


def product(x, w, rs):
    """(exact, tolerance) of one product in the kernels' arithmetic, without the last rounding: x [n, K], w [N, K] and rs
    [N], float64.  A product's accumulations are K / 16 on the longest path and a few sums around them; an x below f16's
    range is off by 2^-38 of the row's largest; the scaling and row_scale round once each."""
    exact = (x @ w.T) * rs
    mag = (np.abs(x) @ np.abs(w).T) * np.abs(rs)
    K = x.shape[1]
    big = np.abs(x).max(-1, keepdims=True) if x.size else np.zeros((x.shape[0], 1))
    tol = mag * (-(-K // 16) + 90) * ACC + big * np.abs(w).sum(-1) * np.abs(rs) * 2.0 ** -38 + np.abs(exact) * 4 * H32
    return exact, tol


def swiglu(h, tol):
    """(exact, tolerance) of silu(h[2n]) h[2n + 1]: silu's slope is at most 1.1; exp, the sum, the quotient and the
    product are off by a few steps of fp32."""
    g, u, eg, eu = h[:, 0::2], h[:, 1::2], tol[:, 0::2], tol[:, 1::2]
    with np.errstate(over="ignore"):
        s = g / (1.0 + np.exp(-g))
    y = s * u
    return y, 1.1 * eg * np.abs(u) + np.abs(s) * eu + 1.1 * eg * eu + np.abs(y) * (16 + np.abs(g)) * H32 * 2 + 2.0 ** -126


def rounded(exact, tol, bf16):
    return tol + (np.abs(exact) + tol) * (HBF if bf16 else H32) + 2.0 ** -133


def adapters(x, a, b, adapter, base, ranks=None, scale=None, split=2.0 ** -16):
    """(exact, tolerance before the last rounding), all float64 but adapter and ranks; split: how far t may be off that
    enters the second product, in two bf16 terms."""
    m, K = x.shape
    L, r, _ = a.shape
    out, tol = base.copy(), np.zeros_like(base)
    for i in range(m):
        l = int(adapter[i])
        if l < 0 or l >= L:
            continue
        n = r if ranks is None else min(max(int(ranks[l]), 0), r)
        s = 1.0 if scale is None else float(scale[l])
        al, bl = a[l, :n], b[l, :, :n]
        t = (al @ x[i]) * s
        # K / 16 accumulations of the first product, its sums over warps and CTAs, the scale; t as bf16 terms
        et = (np.abs(al) @ np.abs(x[i])) * abs(s) * (-(-K // 16) + 24) * ACC + np.abs(t) * split
        delta = bl @ t
        out[i] = base[i] + delta
        tol[i] = np.abs(bl) @ et + (np.abs(bl) @ (np.abs(t) + et)) * (-(-r // 16) * 2 + 4) * ACC + np.abs(out[i]) * 2 * H32
    return out, tol


def logprobs(logits, tokens, inv_temp, n_top):
    """(logprobs, lse, entropy, top_ids, top_logprobs, tolerances of lse / logprobs by |exponent| / entropy); logits
    float64 [rows, V] holding fp32 values."""
    R, V = logits.shape
    c = float(np.float32(inv_temp))
    top = logits.max(-1, keepdims=True)
    empty = top[:, 0] == -np.inf
    d = np.where(logits == -np.inf, -np.inf, (logits - np.where(empty[:, None], 0, top)) * c)
    p = np.exp(d)
    z = p.sum(-1)
    with np.errstate(divide="ignore", invalid="ignore"):
        logz = np.log(z)
        lse = np.where(empty, -np.inf, top[:, 0] * c + logz)
        ent = np.where(empty, 0, logz - (p * np.where(p > 0, d, 0)).sum(-1) / z)
        lp = np.where(empty[:, None], -np.inf, d - logz[:, None])
    got = np.zeros(tokens.shape)
    for i in range(R):
        for j, t in enumerate(tokens[i]):
            got[i, j] = 0.0 if t < 0 else -np.inf if t >= V else lp[i, t]
    ids, vals = np.full((R, n_top), -1, np.int64), np.full((R, n_top), -np.inf)
    for i in range(R):
        o = np.lexsort((np.arange(V), -logits[i]))[:n_top]
        ids[i, :len(o)], vals[i, :len(o)] = o, lp[i, o]
    # a term of the sums: its exponent (three roundings of it) and ex2 (2^-21); a lane adds up to V / 128 of them one after
    # the other, and twenty more; entropy's terms weigh the exponents' errors once more
    seq = (V / 128 + 64) * H32
    dm = np.abs(np.where(np.isfinite(d) & (p > 0), d, 0))
    with np.errstate(invalid="ignore", divide="ignore"):
        es = np.nan_to_num((p * (dm * 4 * H32 + 2.0 ** -21)).sum(-1) / z) + seq
        ee = np.nan_to_num((p * dm * (dm * 4 * H32 + 2.0 ** -20)).sum(-1) / z) + 2 * seq * np.nan_to_num((p * dm).sum(-1) / z)
    el = es + 4 * H32 * (np.abs(np.where(empty, 0, lse)) + np.abs(np.where(empty, 0, logz)) + np.abs(np.where(empty, 0, top[:, 0] * c)) + 1)
    return got, lse, ent, ids, vals, el, es + ee + 4 * H32 * (np.abs(ent) + np.abs(np.where(empty, 0, logz)) + 1)
