"""Operators around a batch's attention step, as a user's program calls them: the experts of a layer, the adapters of
many requests, and what the step answers with.

Kinds of case:
  route     router logits to the k experts of each token, their weights, and the tokens in order of expert;
  grouped   products of the tokens of each expert with its 4-bit weight (E2M1 codes, one E4M3 scale per 16 channels,
            an fp32 scale per output row), ragged numbers of rows, with or without the gated activation;
  combine   the weighted sum of each token's expert outputs, beside a shared expert's output or a residual;
  adapters  low-rank adapters of many requests added beside a shared projection;
  logprobs  log probabilities of given tokens, log-sum-exp, entropy and the likeliest alternatives.

`run` computes the plain forms while `own` is false, and calls the package's operators where it is true.
"""
import math
import random

import torch

own = False

GROUP = 16
DEV = "cuda"
NEG = float("-inf")


def _csa2():
    import compressed_sparse_attention_step_gb300 as c
    return c


# ---------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------
def listed():
    return [
        # the router of one decode step: 64 sequences, 384 experts, six of them active
        dict(name="route_m64_e384", kind="route", m=64, E=384, k=6, bias=True, renorm=True, idle=0.1),
        # a prompt chunk's router
        dict(name="route_m8192_e384", kind="route", m=8192, E=384, k=6, bias=False, renorm=True, idle=0.0),
        # a decode step's experts: one or two rows each, weights are all that counts; gate and up in one product
        dict(name="grouped_m64_e384", kind="grouped", m=64, E=384, k=6, n_in=4096, n_out=2048, act=True, out="bf16",
             skew=0.3, idle=0.0),
        # a small layer of odd sizes, ragged, fp32 result
        dict(name="grouped_m37_e9", kind="grouped", m=37, E=9, k=2, n_in=1040, n_out=1000, act=False, out="fp32",
             skew=1.0, idle=0.1),
        # few experts, many rows each: a prompt chunk whose products bound it
        dict(name="grouped_m4096_e8", kind="grouped", m=4096, E=8, k=2, n_in=4096, n_out=4096, act=True, out="bf16",
             skew=0.3, idle=0.0),
        # the outputs of a decode step's experts beside the shared expert's
        dict(name="combine_m64", kind="combine", m=64, k=6, n=4096, add=True, y="bf16", out="bf16", idle=0.1),
        # a prompt chunk's
        dict(name="combine_m8192", kind="combine", m=8192, k=6, n=4096, add=True, y="bf16", out="bf16", idle=0.0),
        # one request, one adapter: latency
        dict(name="adapters_m1", kind="adapters", m=1, n_in=4096, n_out=4096, r=16, L=4, order="mixed", none=0.0,
             out="bf16"),
        # a decode batch whose requests use 32 adapters, a few none
        dict(name="adapters_m64_l32", kind="adapters", m=64, n_in=4096, n_out=8200, r=32, L=32, order="mixed", none=0.1,
             out="bf16"),
        # a prompt chunk: runs of rows of the same request
        dict(name="adapters_m4100_l8", kind="adapters", m=4100, n_in=8192, n_out=8192, r=64, L=8, order="runs", none=0.1,
             out="bf16"),
        # the answer of one sequence
        dict(name="logprobs_r1", kind="logprobs", rows=1, V=129280, dtype="bf16", n_tok=1, n_top=20, mask=0.0, pad=0,
             inv_temp=1.0),
        # the scores of a long prompt, or of a verify step's nodes: a vocabulary that is no multiple of anything
        dict(name="logprobs_r2048", kind="logprobs", rows=2048, V=129283, dtype="bf16", n_tok=2, n_top=8, mask=0.02,
             pad=13, inv_temp=1.25),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng: random.Random):
    kind = rng.choice(["route", "grouped", "grouped", "combine", "adapters", "adapters", "logprobs", "logprobs"])
    if kind == "route":
        E = _log(rng, 4, 512)
        return dict(kind=kind, m=_log(rng, 1, 8192), E=E, k=rng.randint(1, min(8, E)), bias=rng.random() < 0.5,
                    renorm=rng.random() < 0.5, idle=rng.choice([0.0, 0.1, 0.5]))
    if kind == "grouped":
        E = _log(rng, 1, 384)
        n_in, n_out = 16 * _log(rng, 2, 256), 2 * _log(rng, 8, 2048)
        while E * n_in * n_out > 384 * 4096 * 2048:
            E = max(1, E // 2)
        k = rng.randint(1, min(6, E))
        m = _log(rng, 1, 4096)
        while m * k * n_in * n_out > 8192 * 4096 * 4096:
            m = max(1, m // 2)
        return dict(kind=kind, m=m, E=E, k=k, n_in=n_in, n_out=n_out, act=rng.random() < 0.5,
                    out=rng.choice(["bf16", "bf16", "fp32"]), skew=rng.choice([0.0, 0.3, 1.0, 2.0]),
                    idle=rng.choice([0.0, 0.1]))
    if kind == "combine":
        return dict(kind=kind, m=_log(rng, 1, 8192), k=rng.randint(1, 6), n=_log(rng, 8, 4096), add=rng.random() < 0.5,
                    y=rng.choice(["bf16", "bf16", "fp32"]), out=rng.choice(["bf16", "bf16", "fp32"]),
                    idle=rng.choice([0.0, 0.1, 0.5]))
    if kind == "adapters":
        return dict(kind=kind, m=_log(rng, 1, 4096), n_in=8 * _log(rng, 4, 1024), n_out=_log(rng, 8, 8192),
                    r=rng.choice([8, 16, 24, 32, 64]), L=_log(rng, 1, 64), order=rng.choice(["mixed", "runs"]),
                    none=rng.choice([0.0, 0.1, 0.5]), out=rng.choice(["bf16", "bf16", "fp32"]))
    V = _log(rng, 64, 131072)
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    rows = _log(rng, 1, max(1, min(4096, 2048 * 129283 // V // (1 if dtype == "bf16" else 2))))
    return dict(kind=kind, rows=rows, V=V, dtype=dtype, n_tok=rng.choice([1, 1, 2, 8]),
                n_top=rng.choice([0, 1, 8, 20, 32]), mask=rng.choice([0.0, 0.02, 0.5]), pad=rng.choice([0, 0, 5, 64]),
                inv_temp=rng.choice([1.0, 0.7, 1.25]))


# ---------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------
def _gen(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed * 6271 + 29)
    return g, random.Random(seed * 15485863 + 11)


def _randn(g, shape, dtype=torch.bfloat16, scale=1.0):
    return (torch.randn(shape, generator=g, device=DEV) * scale).to(dtype)


def _quantised(g, rows, C):
    """E2M1 codes [rows, C/2] (even channel in the low nibble) and E4M3 scales [rows, C/16] of N(0, 8^2) weights."""
    codes = torch.empty((rows, C // 2), dtype=torch.uint8, device=DEV)
    scales = torch.empty((rows, C // GROUP), dtype=torch.uint8, device=DEV)
    mids = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=DEV)
    step = max(1, (1 << 26) // C)
    for a in range(0, rows, step):
        b = min(rows, a + step)
        w = torch.randn((b - a, C // GROUP, GROUP), generator=g, device=DEV) * 8.0
        s8 = (w.abs().amax(-1) / 6.0).to(torch.float8_e4m3fn)
        c = torch.bucketize(w.abs() / s8.float()[..., None], mids, out_int32=True).to(torch.uint8)
        c = (c | (torch.signbit(w).to(torch.uint8) << 3)).view(b - a, C)
        codes[a:b] = c[:, 0::2] | (c[:, 1::2] << 4)
        scales[a:b] = s8.view(torch.uint8)
    return codes, scales


def _skewed(g, m, E, skew):
    """Router logits [m, E]: noise, and experts that are chosen more often than others."""
    return torch.randn((m, E), generator=g, device=DEV) + skew * torch.randn((E,), generator=g, device=DEV)


def _idle(g, m, share):
    """int32 [m]: 0 for the padding rows of a batch."""
    return (torch.rand((m,), generator=g, device=DEV) >= share).to(torch.int32)


def _sorted_by_expert(chosen, active, E):
    """chosen int64 [m, k] -> src, offsets, pos, all int32, as the router gives them."""
    m, k = chosen.shape
    flat = torch.where(active[:, None] > 0, chosen, torch.full_like(chosen, E)).reshape(-1)
    order = torch.argsort(flat, stable=True)
    counts = torch.zeros((E + 1,), dtype=torch.int64, device=DEV).scatter_add_(0, flat, torch.ones_like(flat))
    offsets = torch.cat((torch.zeros((1,), dtype=torch.int64, device=DEV), counts[:E].cumsum(0)))
    at = torch.arange(m * k, device=DEV)
    src = torch.where(at < offsets[E], order // k, torch.full_like(order, -1))
    pos = torch.empty_like(order)
    pos[order] = at
    pos = torch.where(pos < offsets[E], pos, torch.full_like(pos, -1)).view(m, k)
    return src.to(torch.int32), offsets.to(torch.int32), pos.to(torch.int32)


def prepare(case, seed):
    g, rnd = _gen(case, seed)
    kind = case["kind"]
    st = {"case": case}
    f32 = torch.float32
    if kind == "route":
        m, E, k = case["m"], case["E"], case["k"]
        st.update(logits=_skewed(g, m, E, 1.0), active=_idle(g, m, case["idle"]),
                  bias=torch.randn((E,), generator=g, device=DEV) if case["bias"] else None,
                  experts=torch.empty((m, k), dtype=torch.int32, device=DEV),
                  weights=torch.empty((m, k), dtype=f32, device=DEV),
                  offsets=torch.empty((E + 1,), dtype=torch.int32, device=DEV),
                  src=torch.empty((m * k,), dtype=torch.int32, device=DEV),
                  pos=torch.empty((m, k), dtype=torch.int32, device=DEV))
        if own:
            c = _csa2()
            st["ws"] = torch.empty((max(1, c.route_workspace_size(m, E)),), dtype=torch.uint8, device=DEV)
    elif kind == "grouped":
        m, E, k, n_in, n_out = (case[n] for n in ("m", "E", "k", "n_in", "n_out"))
        codes, scales = _quantised(g, E * n_out, n_in)
        chosen = torch.topk(_skewed(g, m, E, case["skew"]), k, dim=1).indices
        src, offsets, _ = _sorted_by_expert(chosen, _idle(g, m, case["idle"]), E)
        width = n_out // 2 if case["act"] else n_out
        st.update(x=_randn(g, (m, n_in)), codes=codes.view(E, n_out, -1), scales=scales.view(E, n_out, -1),
                  row_scale=(0.5 + torch.rand((E, n_out), generator=g, device=DEV)) * (n_in ** -0.5 / 8.0),
                  src=src, offsets=offsets, parts=offsets.tolist(),
                  y=torch.zeros((m * k, width), dtype=torch.bfloat16 if case["out"] == "bf16" else f32, device=DEV))
        if own:
            c = _csa2()
            st["packed"] = c.fp4_pack_experts(st["codes"], st["scales"])
            st["ws"] = torch.empty((c.grouped_workspace_size(m * k, n_in),), dtype=torch.uint8, device=DEV)
    elif kind == "combine":
        m, k, n = case["m"], case["k"], case["n"]
        pos = torch.randperm(m * k, generator=g, device=DEV).view(m, k).to(torch.int32)
        pos = torch.where(_idle(g, m, case["idle"])[:, None] > 0, pos, torch.full_like(pos, -1))
        st.update(y=_randn(g, (m * k, n), torch.bfloat16 if case["y"] == "bf16" else f32), pos=pos,
                  weights=torch.softmax(torch.randn((m, k), generator=g, device=DEV), -1),
                  add=_randn(g, (m, n)) if case["add"] else None,
                  out=torch.empty((m, n), dtype=torch.bfloat16 if case["out"] == "bf16" else f32, device=DEV))
    elif kind == "adapters":
        m, n_in, n_out, r, L = (case[n] for n in ("m", "n_in", "n_out", "r", "L"))
        if case["order"] == "mixed":
            which = [rnd.randrange(L) if rnd.random() >= case["none"] else -1 for _ in range(m)]
        else:
            which = []
            while len(which) < m:
                one = rnd.randrange(L) if rnd.random() >= case["none"] else -1
                which += [one] * rnd.randint(1, max(1, min(m, 700)))
            which = which[:m]
        out = torch.bfloat16 if case["out"] == "bf16" else f32
        st.update(x=_randn(g, (m, n_in)), a=_randn(g, (L, r, n_in), scale=n_in ** -0.5), b=_randn(g, (L, n_out, r)),
                  adapter=torch.tensor(which, dtype=torch.int32, device=DEV),
                  ranks=torch.tensor([r if rnd.random() < 0.5 else rnd.randint(1, r) for _ in range(L)],
                                     dtype=torch.int32, device=DEV),
                  scale=0.5 + torch.rand((L,), generator=g, device=DEV), base=_randn(g, (m, n_out), out),
                  out=torch.empty((m, n_out), dtype=out, device=DEV),
                  rows=[(one, torch.tensor([i for i, w in enumerate(which) if w == one], device=DEV))
                        for one in sorted(set(which) - {-1})])
    else:
        R, V = case["rows"], case["V"]
        full = torch.empty((R, V + case["pad"]), dtype=torch.bfloat16 if case["dtype"] == "bf16" else f32, device=DEV)
        step = max(1, (1 << 27) // V)
        for a in range(0, R, step):
            full[a:a + step].normal_(0.0, 3.0, generator=g)
        logits = full[:, :V]
        if case["mask"]:
            for a in range(0, R, step):  # tokens that a grammar rules out
                logits[a:a + step].masked_fill_(torch.rand((min(step, R - a), V), generator=g, device=DEV) < case["mask"], NEG)
            logits[3::7, 5:] = NEG  # rows with a few tokens left
        tokens = torch.randint(0, V, (R, case["n_tok"]), generator=g, device=DEV)
        tokens = torch.where(torch.rand(tokens.shape, generator=g, device=DEV) < 0.05, torch.full_like(tokens, -1), tokens)
        st.update(logits=logits, tokens=tokens.to(torch.int32),
                  logprobs=torch.empty((R, case["n_tok"]), dtype=f32, device=DEV),
                  lse=torch.empty((R,), dtype=f32, device=DEV), entropy=torch.empty((R,), dtype=f32, device=DEV),
                  top_ids=torch.empty((R, case["n_top"]), dtype=torch.int32, device=DEV) if case["n_top"] else None,
                  top_logprobs=torch.empty((R, case["n_top"]), dtype=f32, device=DEV) if case["n_top"] else None)
    return st


# ---------------------------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------------------------
def _dequant(codes, scales):
    v = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
    lut = torch.tensor(v + [-x for x in v], device=codes.device)
    c = torch.stack((lut[(codes & 15).long()], lut[(codes >> 4).long()]), dim=-1).flatten(-2)
    s = scales.view(torch.float8_e4m3fn).to(torch.float32)
    return (c.view(*s.shape, GROUP) * s[..., None]).view(c.shape)


def _route_plain(st):
    case = st["case"]
    k, E = case["k"], case["E"]
    l = st["logits"]
    key = l + st["bias"] if st["bias"] is not None else l
    chosen = torch.sort(key, dim=1, descending=True, stable=True).indices[:, :k]
    p = torch.exp(l - l.amax(1, keepdim=True))
    w = p.gather(1, chosen)
    w = w / (w if case["renorm"] else p).sum(1, keepdim=True)
    on = st["active"][:, None] > 0
    src, offsets, pos = _sorted_by_expert(chosen, st["active"], E)
    return {"experts": torch.where(on, chosen, torch.full_like(chosen, -1)).to(torch.int32),
            "weights": torch.where(on, w, torch.zeros_like(w)), "offsets": offsets, "src": src, "pos": pos}


def _grouped_plain(st):
    case, parts, y = st["case"], st["parts"], st["y"]
    for e in range(case["E"]):
        a, b = parts[e], parts[e + 1]
        if a == b:
            continue
        w = _dequant(st["codes"][e], st["scales"][e]) * st["row_scale"][e][:, None]
        h = torch.matmul(st["x"][st["src"][a:b].long()].float(), w.t())
        if case["act"]:
            gate, up = h[:, 0::2], h[:, 1::2]
            h = gate / (1.0 + torch.exp(-gate)) * up
        y[a:b] = h.to(y.dtype)
    return y


def _combine_plain(st):
    pos = st["pos"].long()
    w = torch.where(pos >= 0, st["weights"], torch.zeros_like(st["weights"]))
    out = st["add"].float() if st["add"] is not None else torch.zeros(st["out"].shape, device=DEV)
    for j in range(pos.shape[1]):
        out = out + w[:, j, None] * st["y"][pos[:, j].clamp(min=0)].float()
    return out.to(st["out"].dtype)


def _adapters_plain(st):
    case = st["case"]
    out = st["base"].float()
    ranks = torch.arange(case["r"], device=DEV)
    for one, rows in st["rows"]:
        keep = ranks < st["ranks"][one]
        a = st["a"][one].float().masked_fill(~keep[:, None], 0.0)
        b = st["b"][one].float().masked_fill(~keep, 0.0)
        t = torch.matmul(st["x"][rows].float(), a.t())
        out[rows] += st["scale"][one] * torch.matmul(t, b.t())
    return out.to(st["base"].dtype)


def _logprobs_plain(st):
    case, n_top = st["case"], st["case"]["n_top"]
    V = case["V"]
    tok = st["tokens"].long()
    got = {"logprobs": [], "lse": [], "entropy": [], "top_ids": [], "top_logprobs": []}
    step = max(1, (1 << 27) // V)
    for a in range(0, case["rows"], step):
        raw = st["logits"][a:a + step].float()
        l = raw * case["inv_temp"]
        m = l.amax(1, keepdim=True)
        empty = m == NEG  # every token ruled out
        d = l - m.masked_fill(empty, 0.0)
        p = torch.exp(d)
        z = p.sum(1, keepdim=True)
        logz = torch.log(z)
        got["lse"].append((m + logz)[:, 0])
        h = logz - (p * d.masked_fill(p == 0, 0.0)).sum(1, keepdim=True) / z
        got["entropy"].append(h.masked_fill(empty, 0.0)[:, 0])
        d = d - logz.masked_fill(empty, 0.0)
        t = tok[a:a + step]
        got["logprobs"].append(torch.where(t >= 0, d.gather(1, t.clamp(min=0)), torch.zeros_like(logz)))
        if n_top:
            # whole numbers in the order of the values (one zero), then of the index, the lowest first
            bits = (raw + 0.0).view(torch.int32).long()
            key = (torch.where(bits < 0, -(bits & 0x7FFFFFFF), bits) << 20) - torch.arange(V, device=DEV)
            ids = torch.topk(key, n_top, dim=1).indices
            got["top_ids"].append(ids.to(torch.int32))
            got["top_logprobs"].append(d.gather(1, ids))
    return {name: torch.cat(v) for name, v in got.items() if v}


def run(state):
    st = state
    case = st["case"]
    kind = case["kind"]
    if kind == "route":
        if not own:
            return _route_plain(st)
        _csa2().csa2_expert_route(st["logits"], st["experts"], st["weights"], st["offsets"], st["src"], st["pos"],
                                  bias=st["bias"], active=st["active"], renorm=case["renorm"], ws=st["ws"])
        return {n: st[n] for n in ("experts", "weights", "offsets", "src", "pos")}
    if kind == "grouped":
        if not own:
            return _grouped_plain(st)
        c = _csa2()
        c.csa2_fp4_grouped(st["x"], st["packed"], st["offsets"], st["y"], src=st["src"], row_scale=st["row_scale"],
                           act=c.ACT_SWIGLU if case["act"] else c.ACT_NONE, ws=st["ws"])
        return st["y"]
    if kind == "combine":
        if not own:
            return _combine_plain(st)
        _csa2().csa2_expert_combine(st["y"], st["pos"], st["weights"], st["out"], add=st["add"])
        return st["out"]
    if kind == "adapters":
        if not own:
            return _adapters_plain(st)
        _csa2().csa2_lora_add(st["x"], st["a"], st["b"], st["adapter"], st["base"], st["out"], ranks=st["ranks"],
                              scale=st["scale"])
        return st["out"]
    if not own:
        return _logprobs_plain(st)
    _csa2().csa2_token_logprobs(st["logits"], st["tokens"], st["logprobs"], lse=st["lse"], entropy=st["entropy"],
                                top_ids=st["top_ids"], top_logprobs=st["top_logprobs"], inv_temp=case["inv_temp"])
    return {n: st[n] for n in ("logprobs", "lse", "entropy", "top_ids", "top_logprobs") if st[n] is not None}


# ---------------------------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------------------------
def work(case):
    kind = case["kind"]
    if kind == "route":
        m, E, k = case["m"], case["E"], case["k"]
        return {"bytes": 4.0 * (m * E + m + E * (2 if case["bias"] else 1) + 4 * m * k), "flops": 2.0 * m * E}
    if kind == "grouped":
        m, E, k, n_in, n_out = (case[n] for n in ("m", "E", "k", "n_in", "n_out"))
        rows = m * k * (1.0 - case["idle"])
        used = E * (1.0 - (1.0 - min(1.0, k / E)) ** m)
        width = n_out // 2 if case["act"] else n_out
        return {"bytes": used * (n_out * n_in * (0.5 + 1.0 / GROUP) + 4.0 * n_out) + 2.0 * m * n_in + 4.0 * (rows + E)
                + rows * width * (2.0 if case["out"] == "bf16" else 4.0), "flops": 2.0 * rows * n_in * n_out}
    if kind == "combine":
        m, k, n = case["m"], case["k"], case["n"]
        rows = m * k * (1.0 - case["idle"])
        return {"bytes": rows * n * (2.0 if case["y"] == "bf16" else 4.0) + 8.0 * m * k + (2.0 * m * n if case["add"] else 0.0)
                + m * n * (2.0 if case["out"] == "bf16" else 4.0), "flops": 2.0 * rows * n}
    if kind == "adapters":
        m, n_in, n_out, r, L = (case[n] for n in ("m", "n_in", "n_out", "r", "L"))
        rows, rank = m * (1.0 - case["none"]), 0.75 * r
        used = L * (1.0 - (1.0 - 1.0 / L) ** rows) if case["order"] == "mixed" else min(L, 1 + rows / 350)
        return {"bytes": rows * n_in * 2.0 + used * rank * (n_in + n_out) * 2.0 + 4.0 * m
                + 2.0 * m * n_out * (2.0 if case["out"] == "bf16" else 4.0), "flops": 2.0 * rows * rank * (n_in + n_out)}
    R, V = case["rows"], case["V"]
    return {"bytes": R * V * (2.0 if case["dtype"] == "bf16" else 4.0) + R * (8.0 * case["n_tok"] + 8.0 + 8.0 * case["n_top"]),
            "flops": 6.0 * R * V}


# ---------------------------------------------------------------------------------------------
# the definitions, in 64 bits (whole numbers for the integer outputs)
# ---------------------------------------------------------------------------------------------
def exact(case, seed):
    kind = case["kind"]
    st = prepare(case, seed)
    f64 = torch.float64
    if kind == "route":
        m, E, k = case["m"], case["E"], case["k"]
        l, active = st["logits"].double(), st["active"].cpu().tolist()
        # what orders the experts is one fp32 sum
        key = (st["logits"] + (st["bias"] if st["bias"] is not None else 0.0)).double()
        best = torch.argsort(-key, dim=1, stable=True)[:, :k]
        w = torch.softmax(l.gather(1, best), 1) if case["renorm"] else torch.softmax(l, 1).gather(1, best)
        lists = [[] for _ in range(E)]
        chosen = best.cpu().tolist()
        for t in range(m):
            if active[t]:
                for j in range(k):
                    lists[chosen[t][j]].append((t, j))
        src, pos, offsets = [-1] * (m * k), [[-1] * k for _ in range(m)], [0]
        for e in range(E):
            for i, (t, j) in enumerate(lists[e]):
                src[offsets[e] + i], pos[t][j] = t, offsets[e] + i
            offsets.append(offsets[e] + len(lists[e]))
        whole = lambda v: torch.tensor(v, dtype=torch.int64, device=DEV)  # noqa: E731
        on = (st["active"] > 0)[:, None]
        return {"experts": torch.where(on, best, torch.full_like(best, -1)), "weights": torch.where(on, w, torch.zeros_like(w)),
                "offsets": whole(offsets), "src": whole(src), "pos": whole(pos)}
    if kind == "grouped":
        n_in, n_out, E = case["n_in"], case["n_out"], case["E"]
        val = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, 0, -.5, -1, -1.5, -2, -3, -4, -6], dtype=f64, device=DEV)
        y = torch.zeros(st["y"].shape, dtype=f64, device=DEV)
        x = st["x"].double()
        for e in range(E):
            at = slice(st["parts"][e], st["parts"][e + 1])
            if at.start == at.stop:
                continue
            w = torch.empty((n_out, n_in), dtype=f64, device=DEV)
            c = st["codes"][e].int()
            w[:, 0::2], w[:, 1::2] = val[c % 16], val[c // 16]
            w *= st["scales"][e].view(torch.float8_e4m3fn).double().repeat_interleave(GROUP, dim=1)
            h = (x[st["src"][at].long()] @ w.T) * st["row_scale"][e].double()
            y[at] = torch.nn.functional.silu(h[:, ::2]) * h[:, 1::2] if case["act"] else h
        return y
    if kind == "combine":
        m, k, n = case["m"], case["k"], case["n"]
        out = st["add"].double() if case["add"] else torch.zeros((m, n), dtype=f64, device=DEV)
        for t0 in range(0, m, 512):
            p = st["pos"][t0:t0 + 512].long()
            rows = st["y"][p.clamp(min=0)].double() * (p >= 0)[..., None]
            out[t0:t0 + 512] += torch.einsum("tk,tkn->tn", st["weights"][t0:t0 + 512].double(), rows)
        return out
    if kind == "adapters":
        out = st["base"].double()
        which = st["adapter"]
        for one in range(case["L"]):
            sel = torch.nonzero(which == one)[:, 0]
            n = int(st["ranks"][one])
            delta = (st["x"][sel].double() @ st["a"][one, :n].double().T) @ st["b"][one, :, :n].double().T
            out[sel] += st["scale"][one].double() * delta
        return out
    R, V, n_top = case["rows"], case["V"], case["n_top"]
    res = {"logprobs": torch.zeros((R, case["n_tok"]), dtype=f64, device=DEV), "lse": torch.empty((R,), dtype=f64, device=DEV),
           "entropy": torch.empty((R,), dtype=f64, device=DEV)}
    if n_top:
        res["top_ids"] = torch.empty((R, n_top), dtype=torch.int64, device=DEV)
        res["top_logprobs"] = torch.empty((R, n_top), dtype=f64, device=DEV)
    for r in range(0, R, 64):
        at = slice(r, min(R, r + 64))
        raw = st["logits"][at].double()
        logp = torch.log_softmax(raw * case["inv_temp"], 1)
        logp = torch.where(raw == NEG, raw, logp)  # (also where every token is ruled out)
        res["lse"][at] = torch.logsumexp(raw * case["inv_temp"], 1)
        res["entropy"][at] = torch.special.entr(logp.exp()).sum(1)
        t = st["tokens"][at].long()
        res["logprobs"][at] = torch.where(t < 0, torch.zeros_like(logp[:, :1]), logp.gather(1, t.clamp(min=0)))
        if n_top:
            order = torch.sort(raw, dim=1, descending=True, stable=True).indices[:, :n_top]
            res["top_ids"][at], res["top_logprobs"][at] = order, logp.gather(1, order)
    return res
