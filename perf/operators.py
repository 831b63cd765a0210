"""Operators of the verify step of drafted tokens over a paged FP4 cache, as a user's program calls them.

Kinds of case:
  tables   block tables and slot maps from request lengths: pages granted to the sequences that grow, taken
           back from those that shrink, and the undo of the same change (drafts granted, then all rejected),
           so that a pass leaves its state as it found it;
  context  the slots of every cache row that a drafted node may select: the committed positions of its
           sequence, then its ancestors and itself;
  append   new main-KV rows quantised to FP4 and new indexer keys copied into the pages' slots;
  tree     attention of a tree of drafted tokens over its nodes' selected FP4 rows, the committed window and
           the drafted ancestors;
  matvec   products of a few token rows with a 4-bit weight (E2M1 codes, one E4M3 scale per 16 channels, an
           fp32 scale per output row).

`run` computes the plain forms while `own` is false, and calls the package's operators where it is true.
"""
import math
import random

import torch

own = False

D, H, DI, GROUP = 512, 16, 128, 16
DEV = "cuda"


def _csa2():
    import compressed_sparse_attention_step_gb300 as c
    return c


# ---------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------
def listed():
    return [
        # one decode step of a serving batch: eight draft slots each, most sequences stay inside a page
        dict(name="tables_draft_b256", kind="tables", B=256, page=64, max_pages=512, n_new=8, mode="draft", spare=600),
        # admission of long prompts, a few requests finishing in the same call
        dict(name="tables_admit_b64", kind="tables", B=64, page=64, max_pages=640, n_new=32768, mode="admit",
             spare=40000),
        # the candidate lists of a verify step, read by the indexer and by the Top-K of every layer
        dict(name="context_b64_n8", kind="context", B=64, N=8, page=64, T=16384),
        # rows of a verify step: 64 sequences, eight drafts each
        dict(name="append_b64_n8", kind="append", rows=512, slots=131072, pad=0.1),
        # a long prompt chunk, with the padding of a ragged batch
        dict(name="append_rows_65500", kind="append", rows=65500, slots=131072, pad=0.03),
        # one sequence, five drafted tokens: latency
        dict(name="tree_b1_n5", kind="tree", B=1, N=5, T=4096, k=512, W=128, pool=True, shape="chain"),
        # a ragged batch with few visible rows, odd sizes, and a cache per sequence instead of pages
        dict(name="tree_b7_n13_k300", kind="tree", B=7, N=13, T=1501, k=300, W=77, pool=False, shape="random"),
        # an ordinary verify step
        dict(name="tree_b64_n8", kind="tree", B=64, N=8, T=8192, k=512, W=128, pool=True, shape="random"),
        # wide trees
        dict(name="tree_b64_n32", kind="tree", B=64, N=32, T=8192, k=512, W=128, pool=True, shape="random"),
        # the latent projection of one token, fp32 result
        dict(name="matvec_m1_n512_k4096", kind="matvec", M=1, N=512, K=4096, out="fp32"),
        # a draft's rows through the query projection, sizes that fill no tile
        dict(name="matvec_m5_n8200_k4112", kind="matvec", M=5, N=8200, K=4112, out="bf16"),
        # the largest weight and batch
        dict(name="matvec_m32_n16384_k8192", kind="matvec", M=32, N=16384, K=8192, out="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng: random.Random):
    kind = rng.choice(["tables", "context", "append", "tree", "tree", "matvec", "matvec"])
    if kind == "tables":
        page = rng.choice([16, 32, 64, 128])
        if rng.random() < 0.5:
            B = _log(rng, 1, 2048)
            return dict(kind=kind, B=B, page=page, max_pages=rng.randint(8, 512), n_new=rng.randint(1, 64), mode="draft",
                        spare=rng.randint(0, 2 * B + 8))
        B = _log(rng, 1, 64)
        n_new = _log(rng, 64, 32768)
        return dict(kind=kind, B=B, page=page, max_pages=n_new // page + rng.randint(2, 64), n_new=n_new, mode="admit",
                    spare=rng.randint(1, 1 + B * (n_new // page + 1)))
    if kind == "context":
        B = _log(rng, 1, 64)
        N = rng.randint(1, max(1, min(64, 512 // B)))
        return dict(kind=kind, B=B, N=N, page=rng.choice([16, 32, 64, 128]), T=_log(rng, 1, 16384))
    if kind == "append":
        return dict(kind=kind, rows=_log(rng, 1, 65500), slots=rng.choice([65536, 100003, 131072]),
                    pad=rng.choice([0.0, 0.05, 0.3]))
    if kind == "tree":
        B = _log(rng, 1, 64)
        N = rng.randint(1, 32)
        return dict(kind=kind, B=B, N=N, T=_log(rng, 1, 8192), k=rng.choice([rng.randint(1, 512), 512]),
                    W=rng.choice([0, rng.randint(1, 128), 128]), pool=rng.random() < 0.5,
                    shape=rng.choice(["chain", "star", "random"]))
    return dict(kind=kind, M=rng.randint(1, 32), N=_log(rng, 4, 16384), K=16 * _log(rng, 4, 512),
                out=rng.choice(["bf16", "fp32"]))


# ---------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------
def _gen(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed * 7919 + 17)
    return g, random.Random(seed * 104729 + 5)


def _e2m1_table(dtype, device):
    v = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
    return torch.tensor(v + [-x for x in v], dtype=dtype, device=device)


def _fp4_rows(x):
    """fp32 rows [r, C] -> E2M1 codes [r, C/2] (even channel in the low nibble) and E4M3 scales [r, C/16]."""
    r, C = x.shape
    xg = x.view(r, C // GROUP, GROUP)
    s8 = (xg.abs().amax(-1) / 6.0).clamp(max=448.0).to(torch.float8_e4m3fn)
    s = s8.to(torch.float32)
    a = xg.abs()
    code = torch.zeros(xg.shape, dtype=torch.uint8, device=x.device)
    # a midpoint counts on equality only where the upper code is even
    for mid, ge in ((0.25, False), (0.75, True), (1.25, False), (1.75, True), (2.5, False), (3.5, True), (5.0, False)):
        t = mid * s[..., None]
        code += (a >= t) if ge else (a > t)
    code |= (torch.signbit(xg).to(torch.uint8) << 3)
    code = torch.where(s[..., None] > 0, code, torch.zeros_like(code)).view(r, C)
    return (code[:, 0::2] | (code[:, 1::2] << 4)).contiguous(), s8.view(torch.uint8)


def _random_fp4(g, rows, C, scale=1.0):
    codes = torch.empty((rows, C // 2), dtype=torch.uint8, device=DEV)
    scales = torch.empty((rows, C // GROUP), dtype=torch.uint8, device=DEV)
    step = max(1, (1 << 25) // C)
    for a in range(0, rows, step):
        b = min(rows, a + step)
        codes[a:b], scales[a:b] = _fp4_rows(torch.randn((b - a, C), generator=g, device=DEV) * scale)
    return codes, scales


def _parents(rnd, B, N, shape):
    rows = []
    for _ in range(B):
        if shape == "chain":
            p = [i - 1 for i in range(N)]
        elif shape == "star":
            p = [-1] * N
        else:
            p = [rnd.randint(-1, i - 1) for i in range(N)]
        rows.append(p)
    return torch.tensor(rows, dtype=torch.int32, device=DEV)


def prepare(case, seed):
    g, rnd = _gen(case, seed)
    kind = case["kind"]
    st = {"case": case}
    if kind == "tables":
        B, P, mp, n_new = case["B"], case["page"], case["max_pages"], case["n_new"]
        old, new = [], []
        for _ in range(B):
            if case["mode"] == "draft":
                o = rnd.randint(0, max(0, mp * P - n_new))
                n = o + (n_new if rnd.random() < 0.9 else rnd.randint(0, n_new))
            elif rnd.random() < 0.2:  # a request that finishes, or loses its rejected tail
                o = rnd.randint(1, mp * P)
                n = rnd.choice([0, rnd.randint(0, o)])
            else:
                o = 0
                n = rnd.randint(1, n_new)
            old.append(o)
            new.append(n)
        held = [-(-o // P) for o in old]
        total = sum(held) + case["spare"]
        perm = torch.randperm(total, generator=g, device=DEV).to(torch.int32)
        table = torch.full((B, mp), -1, dtype=torch.int32, device=DEV)
        at = 0
        for b in range(B):
            table[b, :held[b]] = perm[at:at + held[b]]
            at += held[b]
        room = B * mp + case["spare"]
        free = torch.full((room + 1,), -1, dtype=torch.int32, device=DEV)
        free[:case["spare"]] = perm[at:]
        st.update(old=torch.tensor(old, dtype=torch.int32, device=DEV), new=torch.tensor(new, dtype=torch.int32, device=DEV),
                  table=table, free=free[:room], free_pad=free,
                  pool=torch.tensor([case["spare"], 0, 0, 0], dtype=torch.int32, device=DEV),
                  slots=torch.empty((B, n_new), dtype=torch.int32, device=DEV),
                  granted=torch.empty((B,), dtype=torch.int32, device=DEV),
                  undone=torch.empty((B,), dtype=torch.int32, device=DEV))
    elif kind == "context":
        B, N, P, T = case["B"], case["N"], case["page"], case["T"]
        lens = [rnd.randint(0, T) if rnd.random() < 0.5 else T for _ in range(B)]
        mp = -(-(T + N) // P)
        table = torch.randperm(B * mp, generator=g, device=DEV).to(torch.int32).view(B, mp).contiguous()
        ld = -(-(T + N) // 4) * 4
        st.update(lens=torch.tensor(lens, dtype=torch.int32, device=DEV), table=table,
                  parent=_parents(rnd, B, N, "random"),
                  slots=torch.empty((B * N, ld), dtype=torch.int32, device=DEV),
                  n_slots=torch.empty((B * N,), dtype=torch.int32, device=DEV))
    elif kind == "append":
        n, S = case["rows"], case["slots"]
        slots = torch.randperm(S, generator=g, device=DEV)[:n].to(torch.int32)
        slots = torch.where(torch.rand(n, generator=g, device=DEV) < case["pad"], torch.full_like(slots, -1), slots)
        kv = torch.randn((n, D), generator=g, device=DEV)
        kv = torch.where(torch.rand((n, D), generator=g, device=DEV) < 0.01, kv * 20, kv).to(torch.bfloat16)
        st.update(kv=kv, ki=torch.randn((n, DI), generator=g, device=DEV).to(torch.bfloat16), slots=slots,
                  codes=torch.zeros((S, D // 2), dtype=torch.uint8, device=DEV),
                  scales=torch.zeros((S, D // GROUP), dtype=torch.uint8, device=DEV),
                  KI=torch.zeros((S, DI), dtype=torch.bfloat16, device=DEV))
    elif kind == "tree":
        B, N, T, k, W = case["B"], case["N"], case["T"], case["k"], case["W"]
        codes, scales = _random_fp4(g, B * T, D)
        idx = torch.full((B * N, k), -1, dtype=torch.int32, device=DEV)
        n_valid = torch.zeros((B * N,), dtype=torch.int32, device=DEV)
        perm = torch.randperm(B * T, generator=g, device=DEV) if case["pool"] else None
        take = min(k, T)
        for b in range(B):
            r = torch.rand((N, T), generator=g, device=DEV).topk(take, dim=1).indices.sort(dim=1).values
            if case["pool"]:  # the slots of the sequence's positions
                r = perm[b * T + r]
            idx[b * N:(b + 1) * N, :take] = r.to(torch.int32)
            t = take if rnd.random() < 0.7 else rnd.randint(0, take)
            n_valid[b * N:(b + 1) * N] = t
        n_nodes = [N if rnd.random() < 0.8 else rnd.randint(1, N) for _ in range(B)]
        win = [max(0, W - 1) if rnd.random() < 0.8 else rnd.randint(0, max(0, W - 1)) for _ in range(B)]
        st.update(q=torch.randn((B, N, H, D), generator=g, device=DEV).to(torch.bfloat16),
                  parent=_parents(rnd, B, N, case["shape"]),
                  n_nodes=torch.tensor(n_nodes, dtype=torch.int32, device=DEV),
                  codes=codes if case["pool"] else codes.view(B, T, D // 2),
                  scales=scales if case["pool"] else scales.view(B, T, D // GROUP), idx=idx, n_valid=n_valid,
                  swa=(torch.randn((B, W - 1 + N, D), generator=g, device=DEV).to(torch.bfloat16) if W else None),
                  win_len=torch.tensor(win, dtype=torch.int32, device=DEV),
                  out=torch.zeros((B, N, H, D), dtype=torch.bfloat16, device=DEV),
                  lse=torch.zeros((B, N, H), dtype=torch.float32, device=DEV))
    else:
        M, N, K = case["M"], case["N"], case["K"]
        codes, scales = _random_fp4(g, N, K, 8.0)
        st.update(x=torch.randn((M, K), generator=g, device=DEV).to(torch.bfloat16), codes=codes, scales=scales,
                  row_scale=(0.5 + torch.rand((N,), generator=g, device=DEV)) * (K ** -0.5 / 8.0),
                  y=torch.empty((M, N), dtype=torch.bfloat16 if case["out"] == "bf16" else torch.float32, device=DEV))
        if own:
            c = _csa2()
            st["packed"] = c.fp4_weight_alloc(N, K, device=DEV)
            c.csa2_fp4_pack_weight(codes, scales, st["packed"])
    return st


# ---------------------------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------------------------
def _dequant(codes, scales):
    lut = _e2m1_table(torch.float32, codes.device)
    c = torch.stack((lut[(codes & 15).long()], lut[(codes >> 4).long()]), dim=-1).flatten(-2)
    s = scales.view(torch.float8_e4m3fn).to(torch.float32)
    return (c.view(*s.shape, GROUP) * s[..., None]).view(c.shape)


def _ancestors(parent):
    """[B, N] parents (each below its node, -1: none) -> bool [B, N, N], row i: i and its ancestors; depths."""
    B, N = parent.shape
    a = torch.eye(N, dtype=torch.bool, device=parent.device).expand(B, N, N).clone()
    p = parent.long()
    for i in range(N):
        pi = p[:, i]
        up = a[torch.arange(B, device=a.device), pi.clamp(min=0)] & (pi >= 0)[:, None]
        a[:, i] |= up
    return a, a.sum(-1).to(torch.int32) - 1


def _tables_plain(old, new, P, table, free_pad, pool, slots, granted):
    B, mp = table.shape
    old, new = old.long(), new.long()
    held, want = (old + P - 1) // P, (new + P - 1) // P
    grow = (want - held).clamp(min=0)
    count = pool[0].long()
    # pages given back, in sequence order; the f-th of them is the f-th to be handed out again
    col = torch.arange(mp, device=table.device)[None]
    fits = want <= mp
    shrink = (held - want).clamp(min=0)
    F = shrink.sum()
    f_at = shrink.cumsum(0) - shrink
    back = (col >= want[:, None]) & (col < held[:, None])
    f_idx = f_at[:, None] + col - want[:, None]
    freed = torch.full((B * mp + 1,), -1, dtype=torch.int32, device=table.device)
    freed[torch.where(back, f_idx, torch.full_like(f_idx, B * mp))] = table
    grow = torch.where(fits, grow, torch.zeros_like(grow))
    ok = fits & ((grow == 0) | (grow.cumsum(0) <= count + F))
    got = torch.where(ok, grow, torch.zeros_like(grow))
    A = got.sum()
    a_at = got.cumsum(0) - got
    new_eff = torch.where(ok, new, old)
    a_idx = a_at[:, None] + col - held[:, None]
    take = (col >= held[:, None]) & (col < (held + got)[:, None])
    from_free = free_pad[(count - 1 - (a_idx - F)).clamp(min=0, max=free_pad.numel() - 1)]
    page = torch.where(a_idx < F, freed[a_idx.clamp(min=0, max=B * mp)], from_free)
    table.copy_(torch.where(take, page, table))
    # what is left of the pages given back goes on top of the list
    n_free = free_pad.numel() - 1
    f = torch.arange(B * mp, device=table.device)
    put = torch.where((f >= A) & (f < F), count + F - 1 - f, torch.full_like(f, n_free))
    free_pad[put] = freed[:-1]
    pool[0] = (count + F - A).to(torch.int32)
    if slots is not None:
        i = torch.arange(slots.shape[1], device=table.device)[None]
        pos = old[:, None] + i
        pg = table.long().gather(1, (pos // P).clamp(max=mp - 1))
        slots.copy_(torch.where(pos < new_eff[:, None], pg * P + pos % P, torch.full_like(pos, -1)))
    granted.copy_(new_eff)


def _context_plain(st):
    case = st["case"]
    B, N, P = case["B"], case["N"], case["page"]
    anc, depth = _ancestors(st["parent"])
    lens = st["lens"].long()
    ld = st["slots"].shape[1]
    c = torch.arange(ld, device=lens.device)[None, None]
    order = torch.where(anc, torch.arange(N, device=lens.device)[None, None].expand(B, N, N), N).sort(-1).values
    order = torch.nn.functional.pad(order, (0, ld), value=N)[..., :ld]
    t = c - lens[:, None, None]
    node = order.gather(2, t.clamp(min=0).expand(B, N, ld))
    n = lens[:, None] + depth + 1
    pos = torch.where(t < 0, c, lens[:, None, None] + node)
    page = st["table"].long()[:, None].expand(B, N, -1).gather(2, (pos // P).clamp(max=st["table"].shape[1] - 1))
    st["slots"].copy_(torch.where(c < n[..., None], page * P + pos % P, torch.full_like(pos, -1)).view(B * N, ld))
    st["n_slots"].copy_(n.view(-1))
    return {"slots": st["slots"], "n_slots": st["n_slots"]}


def _append_plain(st):
    ok = st["slots"] >= 0
    S = st["codes"].shape[0]
    at = torch.where(ok, st["slots"].long(), torch.full_like(st["slots"].long(), S))
    codes, scales = _fp4_rows(st["kv"].float())
    for dst, src in ((st["codes"], codes), (st["scales"], scales), (st["KI"], st["ki"])):
        # padding rows land on one row past the end
        full = torch.cat((dst, dst[:1]))
        full[at] = src
        dst.copy_(full[:S])
    return {"codes": st["codes"], "scales": st["scales"], "KI": st["KI"]}


def _tree_plain(st):
    case = st["case"]
    B, N, W, k = case["B"], case["N"], case["W"], case["k"]
    out, lse = st["out"], st["lse"]
    anc, depth = _ancestors(st["parent"])
    live_node = torch.arange(N, device=DEV)[None] < st["n_nodes"][:, None]
    step = max(1, (1 << 27) // (N * k * D))
    for a in range(0, B, step):
        b = min(B, a + step)
        n = b - a
        q = st["q"][a:b].float()
        idx = st["idx"].view(B, N, k)[a:b].long()
        live = (idx >= 0) & (torch.arange(k, device=DEV) < st["n_valid"].view(B, N)[a:b, :, None])
        at = idx.clamp(min=0)
        if case["pool"]:
            rows = _dequant(st["codes"][at], st["scales"][at])
        else:
            sel = torch.arange(a, b, device=DEV)[:, None, None]
            rows = _dequant(st["codes"][sel, at], st["scales"][sel, at])
        s = torch.matmul(q, rows.transpose(-1, -2)) * D ** -0.5
        s = s.masked_fill(~live[:, :, None], float("-inf"))
        if W:
            swa = st["swa"][a:b].float()
            dep = depth[a:b].long()
            r = torch.arange(W - 1, device=DEV)
            lw = (r[None, None] >= dep[..., None]) & (r >= W - 1 - st["win_len"][a:b, None, None])
            ld = anc[a:b] & (dep[:, None, :] > dep[:, :, None] - W)
            lw = torch.cat((lw.expand(n, N, W - 1), ld), -1)
            sw = torch.matmul(q.reshape(n, N * H, D), swa.transpose(-1, -2)).view(n, N, H, -1) * D ** -0.5
            s = torch.cat((s, sw.masked_fill(~lw[:, :, None], float("-inf"))), -1)
        m = s.amax(-1, keepdim=True)
        p = torch.exp(s - torch.where(m == float("-inf"), torch.zeros_like(m), m))
        z = p.sum(-1, keepdim=True)
        o = torch.matmul(p[..., :k], rows)
        if W:
            o = o + torch.matmul(p[..., k:].reshape(n, N * H, -1), swa).view(n, N, H, D)
        o = torch.where(z > 0, o / z, torch.zeros_like(o))
        keep = live_node[a:b, :, None]
        lse[a:b] = torch.where(keep, (m + torch.log(z))[..., 0], lse[a:b])
        out[a:b] = torch.where(keep[..., None], o.to(torch.bfloat16), out[a:b])
    return {"out": out, "lse": lse}


def run(state):
    st = state
    case = st["case"]
    kind = case["kind"]
    if kind == "tables":
        P = case["page"]
        if own:
            c = _csa2()
            c.csa2_block_tables(st["old"], st["new"], P, st["table"], st["free"], st["pool"], st["granted"],
                                slots=st["slots"])
            c.csa2_block_tables(st["granted"], st["old"], P, st["table"], st["free"], st["pool"], st["undone"])
        else:
            _tables_plain(st["old"], st["new"], P, st["table"], st["free_pad"], st["pool"], st["slots"], st["granted"])
            _tables_plain(st["granted"], st["old"], P, st["table"], st["free_pad"], st["pool"], None, st["undone"])
        return {"slots": st["slots"], "granted": st["granted"], "undone": st["undone"], "table": st["table"],
                "free": st["free"], "pool": st["pool"]}
    if kind == "context":
        if own:
            _csa2().csa2_context_slots(st["lens"], st["slots"], st["n_slots"], block_table=st["table"],
                                       page_size=case["page"], parent=st["parent"])
            return {"slots": st["slots"], "n_slots": st["n_slots"]}
        return _context_plain(st)
    if kind == "append":
        if own:
            _csa2().csa2_paged_append(st["slots"], kv_new=st["kv"], codes=st["codes"], scales=st["scales"],
                                      ki_new=st["ki"], KI=st["KI"])
            return {"codes": st["codes"], "scales": st["scales"], "KI": st["KI"]}
        return _append_plain(st)
    if kind == "tree":
        if own:
            _csa2().csa2_tree_attn(st["q"], st["parent"], st["codes"], st["scales"], st["idx"], st["out"],
                                   n_nodes=st["n_nodes"], n_valid=st["n_valid"], swa=st["swa"], win_len=st["win_len"],
                                   W=case["W"], lse=st["lse"])
            return {"out": st["out"], "lse": st["lse"]}
        return _tree_plain(st)
    if own:
        _csa2().csa2_fp4_matvec(st["x"], st["packed"], st["y"], row_scale=st["row_scale"])
        return st["y"]
    w = _dequant(st["codes"], st["scales"]) * st["row_scale"][:, None]
    st["y"].copy_(torch.matmul(st["x"].float(), w.t()))
    return st["y"]


# ---------------------------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------------------------
def work(case):
    kind = case["kind"]
    if kind == "tables":
        B, P = case["B"], case["page"]
        if case["mode"] == "draft":
            pages = min(case["spare"], B * case["n_new"] / P)
        else:
            pages = min(case["spare"] + 0.1 * B * case["max_pages"], 0.8 * B * (case["n_new"] / 2) / P)
        return {"bytes": 4.0 * (B * case["n_new"] + 6 * B + 4 * pages), "flops": 2.0 * B * case["n_new"]}
    if kind == "context":
        B, N, T = case["B"], case["N"], case["T"]
        ld = -(-(T + N) // 4) * 4
        return {"bytes": 4.0 * (B * N * (ld + 1) + B * (N + 1) + B * 0.75 * T / case["page"]), "flops": 2.0 * B * N * ld}
    if kind == "append":
        n = case["rows"] * (1.0 - case["pad"])
        return {"bytes": n * (2 * D + D // 2 + D // GROUP + 4 * DI) + 4.0 * case["rows"], "flops": 8.0 * n * D}
    if kind == "tree":
        B, N, T, k, W = case["B"], case["N"], case["T"], min(case["k"], case["T"]), case["W"]
        nodes, frac = B * N * 0.9, 0.85
        distinct = B * T * (1.0 - (1.0 - frac * k / T) ** (0.9 * N))
        swa = B * (0.9 * max(0, W - 1) + 0.9 * N) * D * 2 if W else 0.0
        per = frac * k + (0.9 * max(0, W - 1) + min(W, 1 + math.log(1 + N)) if W else 0.0)
        return {"bytes": distinct * (D // 2 + D // GROUP) + nodes * (frac * k * 4 + 2 * H * D * 2 + H * 4) + swa,
                "flops": nodes * per * 4.0 * H * D}
    M, N, K = case["M"], case["N"], case["K"]
    return {"bytes": N * K * (0.5 + 1.0 / GROUP) + 4.0 * N + 2.0 * M * K + M * N * (2.0 if case["out"] == "bf16" else 4.0),
            "flops": 2.0 * M * N * K}


# ---------------------------------------------------------------------------------------------
# the definitions, in 64 bits (whole numbers for the integer outputs)
# ---------------------------------------------------------------------------------------------
def _path(parent, i):
    path = []
    while i >= 0:
        path.append(i)
        i = parent[i]
    return path[::-1]


def _exact_tables(old, new, P, mp, table, free, n_free, n_cols):
    """Sequence by sequence: everything that is given back first, then everything that is asked for."""
    B = len(old)
    pages = lambda n: -(-n // P)
    back = []
    for b in range(B):
        back += table[b][pages(new[b]):max(pages(old[b]), pages(new[b]))] if pages(new[b]) < pages(old[b]) else []
    stack = free[:n_free] + back[::-1]
    granted, asked = list(new), 0
    budget = len(stack)
    for b in range(B):
        need = pages(new[b]) - pages(old[b])
        if pages(new[b]) > mp:
            granted[b] = old[b]
        elif need > 0:
            asked += need
            if asked > budget:
                granted[b] = old[b]
            else:
                for j in range(need):
                    table[b][pages(old[b]) + j] = stack.pop()
    free[n_free:len(stack)] = stack[n_free:]
    slots = None
    if n_cols:
        slots = [[table[b][p // P] * P + p % P if p < granted[b] else -1 for p in range(old[b], old[b] + n_cols)]
                 for b in range(B)]
    return granted, slots, len(stack)


def exact(case, seed):
    kind = case["kind"]
    if kind == "tables":
        if case["B"] * case["n_new"] > 4 << 20:
            return None
        st = prepare(case, seed)
        old, new = st["old"].tolist(), st["new"].tolist()
        table, free = st["table"].tolist(), st["free"].tolist()
        P, mp = case["page"], case["max_pages"]
        granted, slots, n = _exact_tables(old, new, P, mp, table, free, case["spare"], case["n_new"])
        undone, _, n = _exact_tables(granted, old, P, mp, table, free, n, 0)
        t = lambda v: torch.tensor(v, dtype=torch.int64, device=DEV)
        return {"slots": t(slots), "granted": t(granted), "undone": t(undone), "table": t(table), "free": t(free),
                "pool": t([n, 0, 0, 0])}
    if kind == "context":
        st = prepare(case, seed)
        P, N = case["page"], case["N"]
        slots = torch.full(st["slots"].shape, -1, dtype=torch.int64, device=DEV)
        ns = []
        for b, L in enumerate(st["lens"].tolist()):
            pos = torch.arange(L, device=DEV)
            tb = st["table"][b].long()
            par = st["parent"][b].tolist()
            for i in range(N):
                p = torch.cat((pos, torch.tensor([L + j for j in _path(par, i)], device=DEV)))
                slots[b * N + i, :p.numel()] = tb[p // P] * P + p % P
                ns.append(p.numel())
        return {"slots": slots, "n_slots": torch.tensor(ns, dtype=torch.int64, device=DEV)}
    if kind == "append":
        # codes, scale bytes and keys are whole numbers fixed by the format: the plain form is their definition
        return None
    if kind == "tree":
        st = prepare(case, seed)
        B, N, W = case["B"], case["N"], case["W"]
        out = torch.zeros((B, N, H, D), dtype=torch.float64, device=DEV)
        lse = torch.zeros((B, N, H), dtype=torch.float64, device=DEV)
        val = _e2m1_table(torch.float64, DEV)
        nn, wl, nv = st["n_nodes"].tolist(), st["win_len"].tolist(), st["n_valid"].view(B, N).tolist()
        for b in range(B):
            par = st["parent"][b].tolist()
            for i in range(nn[b]):
                at = st["idx"][b * N + i, :nv[b][i]].long()
                at = at[at >= 0]
                c = (st["codes"] if case["pool"] else st["codes"][b])[at].int()
                s = (st["scales"] if case["pool"] else st["scales"][b])[at].view(torch.float8_e4m3fn).double()
                v = torch.empty((at.numel(), D), dtype=torch.float64, device=DEV)
                v[:, 0::2], v[:, 1::2] = val[c & 15], val[c >> 4]
                rows = [v * s.repeat_interleave(GROUP, dim=1)]
                if W:
                    path = _path(par, i)
                    d = len(path) - 1
                    rows.append(st["swa"][b, max(d, W - 1 - wl[b]):W - 1].double())
                    rows.append(st["swa"][b, [W - 1 + j for j in path[-W:]]].double())
                rows = torch.cat(rows)
                if rows.shape[0] == 0:
                    lse[b, i] = float("-inf")
                    continue
                sc = st["q"][b, i].double() @ rows.t() / math.sqrt(D)
                lse[b, i] = torch.logsumexp(sc, -1)
                out[b, i] = torch.exp(sc - lse[b, i][:, None]) @ rows
        return {"out": out, "lse": lse}
    st = prepare(case, seed)
    val = _e2m1_table(torch.float64, DEV)
    M, N, K = case["M"], case["N"], case["K"]
    y = torch.empty((M, N), dtype=torch.float64, device=DEV)
    x = st["x"].double()
    for a in range(0, N, 1024):
        c, s = st["codes"][a:a + 1024].int(), st["scales"][a:a + 1024].view(torch.float8_e4m3fn).double()
        w = torch.empty((c.shape[0], K), dtype=torch.float64, device=DEV)
        w[:, 0::2], w[:, 1::2] = val[c & 15], val[c >> 4]
        w *= s.repeat_interleave(GROUP, dim=1)
        y[:, a:a + 1024] = (x @ w.t()) * st["row_scale"][a:a + 1024].double()
    return y
