"""Plain 64-bit forms of the verify step's operators (block tables, context slots, tree attention, 4-bit
products), shared by their tests.  Nothing here uses the library."""
from __future__ import annotations

import numpy as np

import csa2_synth as syn

E2M1 = np.array([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6], np.float64)


def e4m3(b):
    """E4M3FN bytes -> float64."""
    b = np.asarray(b, np.uint8).astype(np.int64)
    e, m, s = (b >> 3) & 15, b & 7, np.where(b & 128, -1.0, 1.0)
    v = np.where(e > 0, (8 + m) * 2.0 ** (e - 10), m * 2.0 ** -9)
    return s * np.where((e == 15) & (m == 7), np.nan, v)


def dequant(codes, scales):
    """codes uint8 [..., C/2], scales uint8 [..., C/16] -> float64 [..., C]."""
    codes = np.asarray(codes)
    v = np.stack((E2M1[codes & 15], E2M1[codes >> 4]), -1).reshape(*codes.shape[:-1], 2 * codes.shape[-1])
    return v * np.repeat(e4m3(scales), 16, -1)


def random_fp4(g, rows, C, lo=0x28, hi=0x48):
    """Random codes and scale bytes (by default scales of 2^-2 .. 2^2)."""
    return (g.integers(0, 256, (rows, C // 2), dtype=np.uint8), g.integers(lo, hi, (rows, C // 16), dtype=np.uint8))


def pages(n, P):
    return -(-n // P)


def block_tables(old, new, P, table, free, n_free, n_new):
    """The definition, sequence by sequence, on Python lists (table and free are changed)."""
    old = [max(o, 0) for o in old]
    new = [max(n, 0) for n in new]
    mp = len(table[0])
    back = []
    for b in range(len(old)):
        back += table[b][pages(new[b], P):pages(old[b], P)]
    stack = free[:n_free] + back[::-1]
    budget, asked, granted = len(stack), 0, list(new)
    grants = []
    for b in range(len(old)):
        need = pages(new[b], P) - pages(old[b], P)
        if need <= 0:
            continue
        if pages(new[b], P) > mp:
            granted[b] = old[b]
            continue
        asked += need
        if asked > budget:
            granted[b] = old[b]
            continue
        grants.append(b)
    for b in grants:
        for j in range(pages(old[b], P), pages(new[b], P)):
            table[b][j] = stack.pop()
    for i in range(n_free, len(stack)):
        free[i] = stack[i]
    slots = [[table[b][p // P] * P + p % P if p < granted[b] else -1 for p in range(old[b], old[b] + n_new)]
             for b in range(len(old))]
    return granted, slots, len(stack)


def path(parent, i):
    """Node i's ancestors and itself, in order of depth."""
    p = []
    while i >= 0:
        p.append(i)
        i = int(parent[i])
    return p[::-1]


def tree_rows(b, i, *, parent, rows, swa, W, win_len):
    """The rows node i attends besides its selected ones: (window rows float64 [n, 512])."""
    if W == 0:
        return np.zeros((0, 512))
    p = path(parent[b], i)
    d = len(p) - 1
    com = swa[b, max(d, W - 1 - int(win_len[b])):W - 1]
    return np.concatenate((com, swa[b, [W - 1 + j for j in p[-W:]]]))


def tree_node(q, sel, win, scale, sel_round=2.0 ** -11):
    """(out, lse, tol of out, tol of lse) of one node: q [16, 512], sel and win rows, all float64.

    The bounds count the roundings of the kernel: P to f16 (2^-11) for selected rows and to bf16 (2^-8) for
    window rows, each score's fp32 sum (8 accumulations of 16 products a warp and 2 sums, at 2^-22 each to
    allow for truncation inside an accumulation), 2^-20 for the exponential and its fp32 argument (up to about
    2^4 at 2^-24), and the output's rounding to bf16 (2^-8).  f16 is spaced by 2^-24 below 2^-14, so there P's
    rounding is off by up to 2^-25 however small P is; the largest P is held at 2^7 or more and belongs to the
    sum, so that is at most 2^-32 of the sum, for each selected row."""
    rows = np.concatenate((sel, win))
    if rows.shape[0] == 0:
        z = np.zeros((16, 512))
        return z, np.full(16, -np.inf), z, np.zeros(16)
    s = q @ rows.T * scale
    es = 10 * 16 * 2.0 ** -22 / 16 * (np.abs(q) @ np.abs(rows).T) * abs(scale) + np.abs(s) * 2.0 ** -22 + 2.0 ** -20
    m = s.max(-1, keepdims=True)
    p = np.exp(s - m)
    lse = (m + np.log(p.sum(-1, keepdims=True)))[:, 0]
    p /= p.sum(-1, keepdims=True)
    d = np.concatenate((np.full(len(sel), sel_round), np.full(len(win), 2.0 ** -8)))
    o = p @ rows
    worst = es.max(-1)
    tol = (p * (d + 2 * worst[:, None])) @ np.abs(rows) + 2.0 ** -8 * np.abs(o) + 2.0 ** -24
    tol = tol + 2.0 ** -32 * np.abs(sel).sum(0)
    return o, lse, tol, worst + 2.0 ** -20 * (1 + np.abs(lse))


def bf16(g, shape, scale=1.0):
    return syn.f32_to_bf16_bits((g.standard_normal(shape) * scale).astype(np.float32))


def f64(bits):
    return syn.bf16_bits_to_f32(bits).astype(np.float64)


def random_parents(g, B, N, shape="random"):
    p = np.full((B, N), -1, np.int32)
    for b in range(B):
        for i in range(1, N):
            p[b, i] = i - 1 if shape == "chain" else -1 if shape == "star" else g.integers(-1, i)
    return p
