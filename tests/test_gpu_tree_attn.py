"""Attention of a tree of drafted tokens against a plain 64-bit form, bound by bound."""
import numpy as np
import pytest

from tests import _verify as V
from tests._cases import bf16_dev, bf16_host, to_dev

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)
import compressed_sparse_attention_step_gb300 as c  # noqa: E402

SCALE = 512 ** -0.5


class Case:
    def __init__(self, seed, B, N, T, k, W, *, pool=True, shape="random", qscale=1.0, full=False):
        g = self.g = np.random.default_rng(seed)
        self.B, self.N, self.T, self.k, self.W, self.pool = B, N, T, k, W, pool
        self.q = V.bf16(g, (B, N, 16, 512), qscale)
        self.codes, self.scales = V.random_fp4(g, B * T, 512)
        self.swa = V.bf16(g, (B, W - 1 + N, 512)) if W else None
        self.parent = V.random_parents(g, B, N, shape)
        self.n_nodes = np.array([N if full or b == 0 else g.integers(0, N + 1) for b in range(B)], np.int32)
        self.win_len = np.array([max(W - 1, 0) if full or b == 0 else g.integers(0, max(W, 1)) for b in range(B)], np.int32)
        self.idx = np.full((B * N, k), -1, np.int32)
        self.n_valid = np.zeros(B * N, np.int32)
        for r in range(B * N):
            n = min(k, T)
            rows = np.sort(g.choice(T, n, replace=False)) + (r // N * T if pool else 0)
            if not full:
                rows = np.where(g.random(n) < 0.05, -1, rows)          # empty entries anywhere
            self.idx[r, :n] = rows
            self.n_valid[r] = k if full or g.random() < 0.5 else g.integers(0, k + 1)

    def dev(self):
        B, T = self.B, self.T
        codes, scales = to_dev(self.codes), to_dev(self.scales)
        if not self.pool:
            codes, scales = codes.view(B, T, 256), scales.view(B, T, 32)
        return dict(q=bf16_dev(self.q), parent=to_dev(self.parent), codes=codes, scales=scales, idx=to_dev(self.idx),
                    n_nodes=to_dev(self.n_nodes), n_valid=to_dev(self.n_valid),
                    swa=bf16_dev(self.swa) if self.W else None, win_len=to_dev(self.win_len), W=self.W,
                    out=torch.full((B, self.N, 16, 512), 9.0, dtype=torch.bfloat16, device="cuda"),
                    lse=torch.full((B, self.N, 16), 9.0, dtype=torch.float32, device="cuda"))

    def check(self, d, scale=SCALE):
        out, lse = V.f64(bf16_host(d["out"])), d["lse"].cpu().numpy().astype(np.float64)
        swa = V.f64(self.swa) if self.W else None
        worst = 0.0
        for b in range(self.B):
            for i in range(self.N):
                if i >= self.n_nodes[b]:                               # left as they were
                    assert (out[b, i] == 9.0).all() and (lse[b, i] == 9.0).all()
                    continue
                r = b * self.N + i
                at = self.idx[r, :self.n_valid[r]]
                at = at[at >= 0]
                base = 0 if self.pool else b * self.T
                sel = V.dequant(self.codes[base + at], self.scales[base + at])
                win = V.tree_rows(b, i, parent=self.parent, rows=None, swa=swa, W=self.W, win_len=self.win_len)
                o, l, tol, tl = V.tree_node(V.f64(self.q[b, i]), sel, win, scale)
                err = np.abs(out[b, i] - o)
                assert (err <= tol).all(), f"b{b} node {i}: worst {np.max(err - tol):.3e} over the bound"
                if sel.shape[0] + win.shape[0]:
                    assert (np.abs(lse[b, i] - l) <= tl).all(), f"b{b} node {i}: lse off by {np.abs(lse[b, i] - l).max():.3e}"
                    worst = max(worst, float((err / np.maximum(tol, 1e-30)).max()))
                else:
                    assert (lse[b, i] == -np.inf).all()
        return worst


@pytest.mark.parametrize("B,N,T,k,W,pool,shape", [
    (1, 1, 1, 1, 1, True, "chain"), (1, 1, 40, 16, 0, True, "chain"), (1, 1, 40, 17, 0, False, "chain"),
    (2, 5, 600, 512, 128, True, "random"), (3, 7, 333, 100, 128, False, "random"), (2, 13, 50, 33, 9, True, "random"),
    (1, 64, 80, 31, 128, True, "chain"), (1, 64, 40, 15, 20, False, "chain"), (2, 20, 64, 48, 3, True, "star"),
    (4, 3, 5, 512, 128, True, "random"), (3, 4, 30, 0, 40, True, "random"), (2, 3, 30, 0, 1, False, "chain"),
    (40, 5, 100, 64, 30, True, "random"), (90, 4, 70, 40, 17, False, "random"),
])
def test_tree_attn(B, N, T, k, W, pool, shape):
    cs = Case(B * 100 + N + W, B, N, T, k, W, pool=pool, shape=shape)
    d = cs.dev()
    c.csa2_device_flags()
    c.csa2_tree_attn(**d)
    assert c.csa2_device_flags() == 0
    cs.check(d)
    first = d["out"].clone(), d["lse"].clone()
    c.csa2_tree_attn(**d)
    assert torch.equal(first[0], d["out"]) and torch.equal(first[1], d["lse"])


def test_no_rows_at_all():
    """Nothing selected and no window: out 0, lse -inf, at both launch forms."""
    for B in (1, 200):
        cs = Case(3, B, 2, 8, 4, 0, full=True)
        cs.n_valid[:] = 0
        d = cs.dev()
        c.csa2_tree_attn(**d)
        assert (d["out"] == 0).all() and (d["lse"] == float("-inf")).all()


@pytest.mark.parametrize("qscale", [2.0 ** -40, 2.0 ** -130, 2.0 ** 20, 1e3])
def test_q_of_any_magnitude(qscale):
    """Q is scaled to f16's range per head: tiny and huge queries, with the softmax scale making up for it."""
    cs = Case(11, 2, 3, 90, 50, 12, qscale=qscale, full=True)
    d = cs.dev()
    scale = float(np.float32(min(SCALE / qscale, 1e38)))
    c.csa2_tree_attn(**d, softmax_scale=scale)
    cs.check(d, scale)


def test_masked_rows_may_hold_anything():
    """NaN and infinities in window rows that a node does not attend, in rows past the batch's nodes and in
    unselected cache rows reach no output."""
    cs = Case(21, 3, 6, 64, 20, 16, shape="star")
    cs.n_nodes[:] = [6, 3, 1]
    cs.win_len[:] = [15, 4, 0]
    d = cs.dev()
    swa = d["swa"]
    for b in range(3):
        swa[b, :15 - int(cs.win_len[b])] = float("nan")
        swa[b, 15 + int(cs.n_nodes[b]):] = float("inf")
    used = np.unique(cs.idx[cs.idx >= 0])
    keep = np.zeros(cs.B * cs.T, bool)
    keep[used] = True
    d["scales"][to_dev(np.flatnonzero(~keep))] = 0x7F                  # E4M3 NaN
    clean = {k: v for k, v in d.items()}
    c.csa2_tree_attn(**clean)
    cs.check(clean)
    # a sibling's drafted row: node i of a star sees itself only
    cs2 = Case(22, 1, 4, 16, 8, 4, shape="star", full=True)
    d2 = cs2.dev()
    c.csa2_tree_attn(**d2)
    ref = d2["out"].clone()
    d2["swa"][0, 3 + 2] = float("nan")
    c.csa2_tree_attn(**d2)
    assert torch.equal(ref[0, [0, 1, 3]], d2["out"][0, [0, 1, 3]]) and torch.isnan(d2["out"][0, 2].float()).all()


def test_index_past_the_cache_is_empty_and_flagged():
    cs = Case(31, 2, 3, 40, 20, 8, full=True)
    d = cs.dev()
    d["idx"][:, 3] = 2 * 40
    d["idx"][:, 5] = 2 ** 31 - 1
    cs.idx[:, 3] = cs.idx[:, 5] = -1
    c.csa2_device_flags()
    c.csa2_tree_attn(**d)
    assert c.csa2_device_flags() == c.FLAG_INDEX_OOB
    cs.check(d)


def test_parents_out_of_order_are_roots_and_flagged():
    cs = Case(32, 1, 5, 40, 20, 16, shape="chain", full=True)
    d = cs.dev()
    d["parent"].copy_(torch.tensor([[0, 4, 1, -9, 3]], dtype=torch.int32))
    cs.parent[:] = [[-1, -1, 1, -1, 3]]
    c.csa2_device_flags()
    c.csa2_tree_attn(**d)
    assert c.csa2_device_flags() == c.FLAG_INDEX_OOB
    cs.check(d)


def test_chain_equals_the_decode_entry_point():
    """A chain is csa2_sparse_attn_decode with Nq queries: the same rows, within both kernels' bounds.  Rows
    here reach 24 and outputs 16, where half a step of bf16 is 2^-8 of 16 = 0.06, so a fixed absolute bound
    does not apply: each side is held to its own roundings (the decode kernels' P to bf16 at worst)."""
    B, N, T, k, W = 3, 6, 700, 512, 128
    cs = Case(41, B, N, T, k, W, pool=False, shape="chain", full=True)
    d = cs.dev()
    c.csa2_tree_attn(**d)
    out, lse = torch.empty_like(d["out"]), torch.empty_like(d["lse"])
    c.csa2_sparse_attn_decode(d["q"], d["codes"], d["scales"], d["idx"], out, n_valid=d["n_valid"], swa=d["swa"],
                              swa_len=torch.full((B,), W - 1 + N, dtype=torch.int32, device="cuda"), W=W, lse=lse)
    cs.check(d)
    a, b = V.f64(bf16_host(d["out"])), V.f64(bf16_host(out))
    for s in range(B):
        for i in range(N):
            at = s * T + cs.idx[s * N + i]
            sel = V.dequant(cs.codes[at], cs.scales[at])
            win = V.tree_rows(s, i, parent=cs.parent, rows=None, swa=V.f64(cs.swa), W=W, win_len=cs.win_len)
            _, _, t1, _ = V.tree_node(V.f64(cs.q[s, i]), sel, win, SCALE)
            _, _, t2, _ = V.tree_node(V.f64(cs.q[s, i]), sel, win, SCALE, sel_round=2.0 ** -8)
            assert (np.abs(a[s, i] - b[s, i]) <= t1 + t2).all()
    assert np.linalg.norm(a - b) <= 1e-2 * np.linalg.norm(b)
    assert float((d["lse"] - lse).abs().max()) <= 1e-2


def test_far_rows_of_a_long_pool():
    """Rows whose byte offset passes 32 bits (16.8 million rows of 256 bytes)."""
    cap, n = (1 << 24) + 4096, 64
    codes = torch.zeros((cap, 256), dtype=torch.uint8, device="cuda")
    scales = torch.zeros((cap, 32), dtype=torch.uint8, device="cuda")
    cs = Case(51, 1, 2, n, n, 5, full=True)
    at = torch.from_numpy(np.sort(np.random.default_rng(1).choice(4000, n, replace=False)) + (1 << 24)).cuda()
    codes[at], scales[at] = to_dev(cs.codes), to_dev(cs.scales)
    d = cs.dev()
    d.update(codes=codes, scales=scales, idx=at[d["idx"].long()].to(torch.int32))
    c.csa2_tree_attn(**d)
    cs.check(d)


def test_captured_and_on_another_stream():
    cs = Case(61, 4, 6, 200, 100, 64)
    d = cs.dev()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        c.csa2_tree_attn(**d)
    s.synchronize()
    cs.check(d)
    ref = d["out"].clone()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            c.csa2_tree_attn(**d)
        graphs.append(g)
    d["out"].fill_(9.0)
    for g in graphs:
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(ref, d["out"])


def test_scores_far_below_zero():
    """Scores of millions, of either sign: the softmax is that of their differences.  Heads whose largest score
    leads by more than both scores' error bounds and 40 attend that row alone (e^-40 is below half of bf16's
    and of fp32's last place), exactly, as an FP4 row is a bf16 row."""
    led = 0
    for sign in (-1.0, 1.0):
        cs = Case(71, 2, 2, 40, 33, 0, full=True)
        d = cs.dev()
        scale = float(np.float32(sign * 1e5))
        c.csa2_tree_attn(**d, softmax_scale=scale)
        out = V.f64(bf16_host(d["out"]))
        for r in range(4):
            q, rows = V.f64(cs.q[r // 2, r % 2]), V.dequant(cs.codes[cs.idx[r]], cs.scales[cs.idx[r]])
            sc = q @ rows.T * scale
            es = 160 * 2.0 ** -22 / 16 * (np.abs(q) @ np.abs(rows).T) * abs(scale) + np.abs(sc) * 2.0 ** -22
            top = np.argsort(sc, -1)[:, ::-1]
            for h in range(16):
                lead = sc[h, top[h, 0]] - sc[h, top[h, 1]]
                if lead > 2 * es[h].max() + 40:
                    led += 1
                    assert np.array_equal(out[r // 2, r % 2, h], rows[top[h, 0]])
    assert led > 100
    # one cache row: P = 1 whatever the score
    cs = Case(72, 1, 1, 1, 1, 0, full=True)
    d = cs.dev()
    for scale in (-1e35, 1e35, 0.0):
        c.csa2_tree_attn(**d, softmax_scale=scale)
        assert np.array_equal(V.f64(bf16_host(d["out"]))[0, 0], np.tile(V.dequant(cs.codes, cs.scales), (16, 1)))


def test_more_nodes_than_run_at_once():
    """Two waves and more of CTAs, a ragged batch."""
    cs = Case(81, 70, 10, 48, 24, 9)
    d = cs.dev()
    c.csa2_tree_attn(**d)
    cs.check(d)


def test_two_calls_at_once():
    """Two streams, different inputs."""
    a, b = Case(91, 3, 9, 90, 70, 33), Case(92, 30, 6, 60, 40, 20, pool=False)
    da, db = a.dev(), b.dev()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for s in (s1, s2):
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(20):
        c.csa2_tree_attn(**da, stream=s1)
        c.csa2_tree_attn(**db, stream=s2)
    torch.cuda.synchronize()
    a.check(da)
    b.check(db)


def test_tree_attn_in_place_and_an_empty_pool():
    """out may be q (at each number of CTAs a node); with a pool of no rows every entry is empty."""
    g = torch.Generator(device="cuda").manual_seed(3)
    for B, N, k in ((1, 5, 64), (7, 5, 64), (40, 8, 64)):
        q = torch.randn((B, N, 16, 512), generator=g, device="cuda").bfloat16()
        parent = torch.arange(-1, N - 1, device="cuda", dtype=torch.int32).repeat(B, 1)
        codes = torch.randint(0, 256, (300, 256), generator=g, device="cuda", dtype=torch.uint8)
        scales = torch.randint(40, 60, (300, 32), generator=g, device="cuda", dtype=torch.uint8)
        idx = torch.randint(0, 300, (B * N, k), generator=g, device="cuda", dtype=torch.int32)
        swa = torch.randn((B, 7 + N, 512), generator=g, device="cuda").bfloat16()
        out = torch.empty_like(q)
        c.csa2_tree_attn(q, parent, codes, scales, idx, out, swa=swa, W=8)
        same = q.clone()
        c.csa2_tree_attn(same, parent, codes, scales, idx, same, swa=swa, W=8)
        assert torch.equal(out, same)
        none, some = torch.empty_like(q), torch.empty_like(q)
        c.csa2_device_flags()
        c.csa2_tree_attn(q, parent, codes, scales, torch.full_like(idx, -1), some, swa=swa, W=8)
        c.csa2_tree_attn(q, parent, codes[:0], scales[:0], torch.full_like(idx, -1), none, swa=swa, W=8)
        assert c.csa2_device_flags() == 0 and torch.equal(none, some)
        c.csa2_tree_attn(q, parent, codes[:0], scales[:0], idx, none, swa=swa, W=8)
        assert c.csa2_device_flags() == c.FLAG_INDEX_OOB and torch.equal(none, some)


SMS = torch.cuda.get_device_properties(0).multi_processor_count


@pytest.mark.parametrize("rest,N,k", [(1, 1, 12), (19, 1, 20), (38, 2, 9), (40, 4, 260), (94, 2, 256), (100, 4, 30)])
def test_a_few_nodes_behind_the_last_full_wave(rest, N, k):
    """Just more nodes than run at once: the last ones go to a second launch."""
    B = -(-(3 * SMS + rest) // N)
    cs = Case(rest, B, N, k + 5, k, 7)
    cs.n_nodes[:] = N
    d = cs.dev()
    d["n_nodes"] = None
    c.csa2_tree_attn(**d)
    cs.check(d)


@pytest.mark.parametrize("captured", [False, True])
def test_two_launches_are_one_to_what_comes_next(captured):
    """Each call's queries are the last call's outputs, with nothing between the calls, eager and captured: the
    same bits as with a synchronisation after each."""
    B, N = -(-(3 * SMS + 20) // 4), 4
    cs = Case(21, B, N, 60, 48, 9, full=True)
    d = cs.dev()
    del d["out"], d["n_nodes"]
    a, b, keep = (torch.empty_like(d["q"]) for _ in range(3))
    x = d.pop("q")

    def chain(sync):
        src = x
        for i in range(6):
            dst = (a, b)[i & 1]
            c.csa2_tree_attn(q=src, out=dst, **d, softmax_scale=4.0)
            if sync:
                torch.cuda.synchronize()
            src = dst
        return src
    keep.copy_(chain(True))
    assert torch.isfinite(keep.float()).all() and not torch.equal(keep, x)
    run = lambda: chain(False)  # noqa: E731
    if captured:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            run()
        run = lambda: graph.replay() or b  # noqa: E731
    for _ in range(20):
        a.fill_(3.0), b.fill_(5.0)
        assert torch.equal(run(), keep)


def test_queries_and_caches_past_32_bits():
    """The last nodes of a call whose queries, and whose caches of a sequence each, pass 4 GB together."""
    B, N, cap, k = 4200, 64, 4096, 24
    g = torch.Generator(device="cuda").manual_seed(4)
    q = torch.zeros((B, N, 16, 512), dtype=torch.bfloat16, device="cuda")
    codes = torch.zeros((B, cap, 256), dtype=torch.uint8, device="cuda")
    scales = torch.zeros((B, cap, 32), dtype=torch.uint8, device="cuda")
    q[-2:] = torch.randn((2, N, 16, 512), generator=g, device="cuda").bfloat16()
    codes[-2:] = torch.randint(0, 256, (2, cap, 256), generator=g, device="cuda", dtype=torch.uint8)
    scales[-2:] = torch.randint(0x28, 0x48, (2, cap, 32), generator=g, device="cuda", dtype=torch.uint8)
    parent = torch.full((B, N), -1, dtype=torch.int32, device="cuda")
    idx = torch.randint(0, cap, (B * N, k), generator=g, device="cuda", dtype=torch.int32)
    out = torch.full_like(q, 9.0)
    assert q.numel() * 2 > 2 ** 32 and codes.numel() > 2 ** 32
    c.csa2_tree_attn(q, parent, codes, scales, idx, out)
    near = torch.full_like(q[-2:], 9.0)
    c.csa2_tree_attn(q[-2:].contiguous(), parent[-2:], codes[-2:], scales[-2:], idx[-2 * N:], near)
    assert torch.equal(out[-2:], near) and bool((out[:-2] == 0).all())


@pytest.mark.parametrize("rest,N,k,W", [(1, 1, 320, 0), (19, 1, 313, 7), (38, 2, 300, 20), (72, 4, 512, 3)])
def test_many_rows_for_a_few_nodes_behind_the_last_full_wave(rest, N, k, W):
    """As above with as many rows as make a second launch worth it."""
    B = (3 * SMS + rest) // N
    assert 2 * (B * N - 3 * SMS) <= SMS and k + W >= 320
    cs = Case(rest, B, N, k + 5, k, W)
    cs.n_nodes[:] = N
    d = cs.dev()
    d["n_nodes"] = None
    c.csa2_device_flags()
    c.csa2_tree_attn(**d)
    assert c.csa2_device_flags() == 0
    cs.check(d)


@pytest.mark.parametrize("captured", [False, True])
def test_two_launches_of_many_rows_are_one_to_what_comes_next(captured):
    """Each call's queries and lists are what the calls before it wrote, with nothing between them."""
    B, N = (3 * SMS + 40) // 4, 4
    cs = Case(23, B, N, 400, 330, 9, full=True)
    d = cs.dev()
    del d["out"], d["n_nodes"]
    a, b, keep = (torch.empty_like(d["q"]) for _ in range(3))
    x, idx = d.pop("q"), d.pop("idx")
    lists = torch.full_like(idx, -1)

    def chain(sync):
        src = x
        lists.fill_(-1)
        for i in range(6):
            lists[:, 50 * i:50 * i + 60].copy_(idx[:, 50 * i:50 * i + 60])      # the lists grow behind every call
            dst = (a, b)[i & 1]
            c.csa2_tree_attn(q=src, out=dst, idx=lists, **d, softmax_scale=4.0)
            if sync:
                torch.cuda.synchronize()
            src = dst
        return src
    keep.copy_(chain(True))
    assert torch.isfinite(keep.float()).all() and not torch.equal(keep, x)
    run = lambda: chain(False)  # noqa: E731
    if captured:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            run()
        run = lambda: graph.replay() or b  # noqa: E731
    for _ in range(20):
        a.fill_(3.0), b.fill_(5.0)
        assert torch.equal(run(), keep)


def _half_step(x):
    """Half the spacing of bf16 at |x| (8 significant bits)."""
    return 2.0 ** (np.floor(np.log2(np.maximum(np.abs(x), 2.0 ** -126))) - 8)


@pytest.mark.parametrize("B,N,W,shape", [(2, 3, 128, "chain"), (3, 20, 128, "random"), (30, 4, 128, "random"),
                                         (130, 4, 60, "star"), (1, 64, 128, "chain"), (2, 5, 1, "chain")])
def test_window_rows_are_weighed_in_32_bits_but_for_the_output(B, N, W, shape):
    """Window rows alone: the output is the exact value's own bf16 rounding but for P held in two bf16 terms (2^-16:
    half a step of the first, 2^-8, times half a step of the second), the scores' and exponentials' errors (as in
    V.tree_node, twice: numerator and sum) and 40 accumulations at 2^-22 (12 steps of two products, the merge of
    eight parts, the division)."""
    cs = Case(B + N + W, B, N, 4, 0, W, shape=shape)
    d = cs.dev()
    c.csa2_tree_attn(**d)
    cs.check(d)
    out, swa = V.f64(bf16_host(d["out"])), V.f64(cs.swa)
    for b in range(B):
        for i in range(int(cs.n_nodes[b])):
            rows = V.tree_rows(b, i, parent=cs.parent, rows=None, swa=swa, W=W, win_len=cs.win_len)
            q = V.f64(cs.q[b, i])
            s = q @ rows.T * SCALE
            es = (10 * 2.0 ** -22 * (np.abs(q) @ np.abs(rows).T) * SCALE + np.abs(s) * 2.0 ** -22 + 2.0 ** -20).max(-1)
            p = np.exp(s - s.max(-1, keepdims=True))
            p /= p.sum(-1, keepdims=True)
            o = p @ rows
            e = (p * (2.0 ** -16 + 2 * es[:, None] + 40 * 2.0 ** -22)) @ np.abs(rows)
            err = np.abs(out[b, i] - o)
            tol = e + _half_step(np.abs(o) + e)
            assert (err <= tol).all(), f"b{b} node {i}: {(err > tol).sum()} of {err.size}, {np.max(err - tol):.3e} over"


# how many CTAs share a node goes by the nodes and by the rows that their lists may hold (k + W): at 128 and 256 rows,
# at an eighth, a quarter and five eighths of the SMs, on both sides; fewer steps of 16 rows than CTAs among them
@pytest.mark.parametrize("n", [SMS // 8, SMS // 8 + 1, SMS // 4, SMS // 4 + 1, 5 * SMS // 8, 5 * SMS // 8 + 1])
@pytest.mark.parametrize("k,W", [(127, 0), (0, 127), (128, 0), (120, 8), (0, 128), (128, 127), (250, 6), (512, 0)])
def test_a_node_shared_by_some_ctas(n, k, W):
    cs = Case(n + k, n, 1, 600, k, W)
    cs.n_nodes[:] = 1
    cs.n_valid[n // 2:] = np.minimum(cs.n_valid[n // 2:], np.arange(n - n // 2) % 40)     # short lists, empty ones
    d = cs.dev()
    c.csa2_device_flags()
    c.csa2_tree_attn(**d)
    assert c.csa2_device_flags() == 0
    cs.check(d)


@pytest.mark.parametrize("B,N", [(1, 5), (7, 4), (19, 5)])
def test_shared_nodes_without_rows_and_in_place(B, N):
    """Eight and four CTAs a node: nothing selected gives out 0 and lse -inf; out may be q."""
    assert B * N * 8 <= 5 * SMS
    cs = Case(B, B, N, 700, 512, 0, full=True)
    d = cs.dev()
    d["n_valid"].zero_()
    c.csa2_tree_attn(**d)
    assert (d["out"] == 0).all() and (d["lse"] == float("-inf")).all()
    cs = Case(B + 1, B, N, 700, 300, 40, full=True)
    d = cs.dev()
    c.csa2_tree_attn(**d)
    cs.check(d)
    same = d["q"].clone()
    c.csa2_tree_attn(**{**d, "q": same, "out": same})
    assert torch.equal(same, d["out"])
    empty = {**d, "codes": d["codes"][:0], "scales": d["scales"][:0]}
    some, none = torch.empty_like(same), torch.empty_like(same)
    c.csa2_device_flags()
    c.csa2_tree_attn(**{**d, "idx": torch.full_like(d["idx"], -1), "out": some})
    assert c.csa2_device_flags() == 0
    c.csa2_tree_attn(**{**empty, "out": none})
    assert c.csa2_device_flags() == c.FLAG_INDEX_OOB and torch.equal(some, none)


@pytest.mark.parametrize("scale", [-1e5, 1e5])
def test_scores_far_from_zero_at_shared_nodes(scale):
    """A row that leads by more than all errors and 40 is attended alone, whichever CTA of a node holds it."""
    cs = Case(74, 2, 2, 200, 190, 0, full=True)
    d = cs.dev()
    s32 = float(np.float32(scale))
    c.csa2_tree_attn(**d, softmax_scale=s32)
    out, led = V.f64(bf16_host(d["out"])), 0
    for r in range(4):
        q, rows = V.f64(cs.q[r // 2, r % 2]), V.dequant(cs.codes[cs.idx[r]], cs.scales[cs.idx[r]])
        sc = q @ rows.T * s32
        es = 10 * 2.0 ** -22 * (np.abs(q) @ np.abs(rows).T) * abs(s32) + np.abs(sc) * 2.0 ** -22
        top = np.argsort(sc, -1)[:, ::-1]
        for h in range(16):
            if sc[h, top[h, 0]] - sc[h, top[h, 1]] > 2 * es[h].max() + 40:
                led += 1
                assert np.array_equal(out[r // 2, r % 2, h], rows[top[h, 0]])
    assert led > 20


def test_a_few_nodes_behind_two_waves():
    B, N, k, W = (6 * SMS + 30) // 6, 6, 500, 12
    cs = Case(77, B, N, k + 3, k, W)
    cs.n_nodes[:] = N
    d = cs.dev()
    d["n_nodes"] = None
    c.csa2_tree_attn(**d)
    cs.check(d)
