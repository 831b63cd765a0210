"""The operators of a layer around a verify step, run together: attention of the drafted nodes, the shared 4-bit
projection with its requests' adapters, the router, the experts' products and their sum, and the log probabilities of the
drafted children.  Every stage is checked against its 64-bit form on what the stage before it gave; the whole is captured
into a graph and replayed on other requests."""
import numpy as np
import pytest

from tests import _layer as P
from tests import _verify as V
from tests._cases import bf16_dev, to_dev

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)
import compressed_sparse_attention_step_gb300 as c  # noqa: E402

B, N, T, K_SEL, W = 5, 4, 300, 96, 24
HID, E, K, WIDTH, VOC, L, R, KIDS = 256, 24, 3, 144, 1003, 4, 16, 2
M, ATT = B * N, 16 * 512


def host(t):
    return t.float().cpu().numpy().astype(np.float64) if t.is_floating_point() else t.cpu().numpy()


def packed(g, n_out, n_in, lo=0x28, hi=0x40):
    codes, scales = V.random_fp4(g, n_out, n_in, lo, hi)
    p = c.fp4_weight_alloc(n_out, n_in)
    c.csa2_fp4_pack_weight(to_dev(codes), to_dev(scales), p)
    return p, V.dequant(codes, scales)


def experts(g, n_out, n_in):
    codes, scales = V.random_fp4(g, E * n_out, n_in, 0x28, 0x40)
    p = c.fp4_pack_experts(to_dev(codes).view(E, n_out, -1), to_dev(scales).view(E, n_out, -1))
    return p, V.dequant(codes, scales).reshape(E, n_out, n_in)


def scales_of(g, shape, n_in):
    return ((0.5 + g.random(shape)) * (n_in ** -0.5 / 2)).astype(np.float32)


class Step:
    """The weights of a layer, and the buffers of a batch of requests."""

    def __init__(self):
        g = np.random.default_rng(77)
        self.proj, self.w_proj = packed(g, HID, ATT)
        self.rs_proj = scales_of(g, HID, ATT)
        self.up, self.w_up = experts(g, 2 * WIDTH, HID)
        self.rs_up = scales_of(g, (E, 2 * WIDTH), HID)
        self.down, self.w_down = experts(g, HID, WIDTH)
        self.rs_down = scales_of(g, (E, HID), WIDTH)
        self.head, self.w_head = packed(g, VOC, HID)
        self.rs_head = scales_of(g, VOC, HID)
        self.a, self.b = V.bf16(g, (L, R, ATT), ATT ** -0.5), V.bf16(g, (L, HID, R))
        self.lora_scale = g.random(L).astype(np.float32)
        self.w_router = torch.from_numpy(g.standard_normal((HID, E)).astype(np.float32)).cuda()
        self.bias = g.standard_normal(E).astype(np.float32) * 0.1
        dev = lambda x: to_dev(x)  # noqa: E731
        self.d = dict(rs_proj=dev(self.rs_proj), rs_up=dev(self.rs_up), rs_down=dev(self.rs_down), rs_head=dev(self.rs_head),
                      a=bf16_dev(self.a), b=bf16_dev(self.b), lora_scale=dev(self.lora_scale), bias=dev(self.bias))
        i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")  # noqa: E731
        bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
        f32 = lambda *s: torch.zeros(s, device="cuda")  # noqa: E731
        self.q, self.parent, self.n_nodes = bf(B, N, 16, 512), i32(B, N), i32(B)
        self.codes, self.scales = (torch.zeros((B, T, n), dtype=torch.uint8, device="cuda") for n in (256, 32))
        self.idx, self.swa = i32(M, K_SEL), bf(B, W - 1 + N, 512)
        self.adapter, self.active, self.tokens = i32(M), i32(M), i32(M, KIDS)
        self.att, self.h, self.hl = bf(B, N, 16, 512), bf(M, HID), bf(M, HID)
        self.rl = f32(M, E)
        self.route = i32(M, K), f32(M, K), i32(E + 1), i32(M * K), i32(M, K)
        self.z, self.y, self.o = bf(M * K, WIDTH), bf(M * K, HID), bf(M, HID)
        self.logits, self.lp, self.ent = f32(M, VOC), f32(M, KIDS), f32(M)
        self.top, self.top_lp = i32(M, 5), f32(M, 5)
        size = max(c.grouped_workspace_size(M * K, HID), c.grouped_workspace_size(M * K, WIDTH))
        self.ws = torch.empty(size, dtype=torch.uint8, device="cuda")

    def requests(self, seed):
        g = np.random.default_rng(seed)
        self.att.zero_()  # (outputs of padding nodes are left as they were)
        self.q.copy_(bf16_dev(V.bf16(g, (B, N, 16, 512))))
        self.parent.copy_(to_dev(V.random_parents(g, B, N)))
        nodes = g.integers(1, N + 1, B).astype(np.int32)
        self.n_nodes.copy_(to_dev(nodes))
        codes, scales = V.random_fp4(g, B * T, 512)
        self.codes.copy_(to_dev(codes).view(B, T, -1))
        self.scales.copy_(to_dev(scales).view(B, T, -1))
        self.idx.copy_(to_dev(np.stack([np.sort(g.choice(T, K_SEL, replace=False)) for _ in range(M)]).astype(np.int32)))
        self.swa.copy_(bf16_dev(V.bf16(g, (B, W - 1 + N, 512))))
        self.adapter.copy_(to_dev(np.repeat(g.integers(-1, L, B), N).astype(np.int32)))
        self.active.copy_(to_dev((np.arange(N)[None] < nodes[:, None]).astype(np.int32).reshape(-1)))
        self.tokens.copy_(to_dev(g.integers(-1, VOC, (M, KIDS)).astype(np.int32)))

    def run(self):
        d = self.d
        c.csa2_tree_attn(self.q, self.parent, self.codes, self.scales, self.idx, self.att, n_nodes=self.n_nodes, swa=self.swa, W=W)
        x = self.att.view(M, ATT)
        c.csa2_fp4_matvec(x, self.proj, self.h, row_scale=d["rs_proj"])
        c.csa2_lora_add(x, d["a"], d["b"], self.adapter, self.h, self.hl, scale=d["lora_scale"])
        torch.matmul(self.hl.float(), self.w_router, out=self.rl)
        c.csa2_expert_route(self.rl, *self.route, bias=d["bias"], active=self.active, scale=2.5)
        experts_, weights, offsets, src, pos = self.route
        c.csa2_fp4_grouped(self.hl, self.up, offsets, self.z, src=src, row_scale=d["rs_up"], act=c.ACT_SWIGLU, ws=self.ws)
        c.csa2_fp4_grouped(self.z, self.down, offsets, self.y, row_scale=d["rs_down"], ws=self.ws)
        c.csa2_expert_combine(self.y, pos, weights, self.o, add=self.hl)
        c.csa2_fp4_matvec(self.o, self.head, self.logits, row_scale=d["rs_head"])
        c.csa2_token_logprobs(self.logits, self.tokens, self.lp, entropy=self.ent, top_ids=self.top, top_logprobs=self.top_lp)

    def outputs(self):
        return [t.clone() for t in (self.h, self.hl, *self.route, self.o, self.logits, self.lp, self.ent, self.top, self.top_lp)]

    def check(self):
        near = lambda got, exact, tol, what: (np.abs(host(got) - exact) <= tol).all() or pytest.fail(what)  # noqa: E731
        x = host(self.att.view(M, ATT))
        exact, tol = P.product(x, self.w_proj, self.rs_proj.astype(np.float64))
        near(self.h, exact, P.rounded(exact, tol, True), "projection")
        exact, tol = P.adapters(x, V.f64(self.a), V.f64(self.b), host(self.adapter), host(self.h), None, self.lora_scale)
        near(self.hl, exact, P.rounded(exact, tol, True), "adapters")
        rl = self.rl.cpu().numpy()
        want = P.route(rl, K, self.bias, host(self.active), scale=2.5)
        for got, ref, what in zip(self.route, want, ("experts", "weights", "offsets", "src", "pos")):
            if what == "weights":
                near(got, ref, P.route_tol(rl, ref), what)
            else:
                assert np.array_equal(host(got), ref), what
        offsets, src, pos = want[2], want[3], want[4]
        hl, z, y = host(self.hl), host(self.z), host(self.y)
        for e in range(E):
            a, b = offsets[e], offsets[e + 1]
            exact, tol = P.swiglu(*P.product(hl[src[a:b]], self.w_up[e], self.rs_up[e].astype(np.float64)))
            near(self.z[a:b], exact, P.rounded(exact, tol, True), f"expert {e} up")
            exact, tol = P.product(z[a:b], self.w_down[e], self.rs_down[e].astype(np.float64))
            near(self.y[a:b], exact, P.rounded(exact, tol, True), f"expert {e} down")
        w = host(self.route[1])
        terms = np.where((pos >= 0)[..., None], w[..., None] * y[np.maximum(pos, 0)], 0)
        exact = hl + terms.sum(1)
        near(self.o, exact, P.rounded(exact, (np.abs(hl) + np.abs(terms).sum(1)) * (K + 1) * P.H32 * 2, True), "sum")
        exact, tol = P.product(host(self.o), self.w_head, self.rs_head.astype(np.float64))
        near(self.logits, exact, P.rounded(exact, tol, False), "logits")
        lp, _, ent, ids, vals, el, ee = P.logprobs(host(self.logits), host(self.tokens), 1.0, 5)
        near(self.lp, lp, el[:, None] + 4 * P.H32 * np.abs(lp), "logprobs")
        near(self.ent, ent, ee + 4 * P.H32 * np.abs(ent), "entropy")
        assert np.array_equal(host(self.top), ids)
        near(self.top_lp, vals, el[:, None] + 4 * P.H32 * np.abs(vals), "top_logprobs")


def test_layer_step_eager_and_replayed():
    s = Step()
    eager = {}
    for seed in (1, 2, 3):
        s.requests(seed)
        s.run()
        torch.cuda.synchronize()
        s.check()
        eager[seed] = s.outputs()
    assert c.csa2_device_flags() == 0
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.run()
    for seed in (2, 3, 1, 2):
        s.requests(seed)
        graph.replay()
        torch.cuda.synchronize()
        for got, want in zip(s.outputs(), eager[seed]):
            assert torch.equal(got, want)
    assert c.csa2_device_flags() == 0
