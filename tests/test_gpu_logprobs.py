"""Log probabilities, log-sum-exp, entropy and the likeliest tokens against a plain 64-bit form."""
import numpy as np
import pytest

from tests import _layer as P
from tests._cases import to_dev

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)
import compressed_sparse_attention_step_gb300 as c  # noqa: E402

INF = float("inf")


def host(t):
    return t.float().cpu().numpy().astype(np.float64) if t.is_floating_point() else t.cpu().numpy()


def check(logits, tokens, inv_temp=1.0, n_top=0):
    """logits: a tensor [rows, V] on the GPU, whose rows may be apart."""
    R, n_tok = logits.shape[0], tokens.shape[1]
    f = lambda *s: torch.full(s, 9.0, device="cuda")  # noqa: E731
    lp, lse, ent, tl = f(R, n_tok), f(R), f(R), f(R, n_top)
    ti = torch.full((R, n_top), 9, dtype=torch.int32, device="cuda")
    c.csa2_token_logprobs(logits, to_dev(tokens), lp, lse=lse, entropy=ent, top_ids=ti if n_top else None,
                          top_logprobs=tl if n_top else None, inv_temp=inv_temp)
    want = P.logprobs(host(logits), tokens, inv_temp, n_top)
    el, ee = want[5], want[6]

    def near(a, b, tol, what):
        a, tol = host(a), np.broadcast_to(tol, b.shape)
        assert np.array_equal(np.isfinite(a), np.isfinite(b)) and np.array_equal(a[~np.isfinite(b)], b[~np.isfinite(b)]), what
        ok = np.isfinite(b)
        assert (np.abs(a[ok] - b[ok]) <= tol[ok] + 4 * P.H32 * np.abs(b[ok])).all(), what
    near(lse, want[1], el, "lse")
    near(lp, want[0], el[:, None], "logprobs")
    near(ent, want[2], ee, "entropy")
    if n_top:
        assert np.array_equal(host(ti), want[3])
        near(tl, want[4], el[:, None], "top_logprobs")
    return lp, lse, ent, ti, tl


def draw(g, R, V, dtype, scale=3.0):
    return torch.from_numpy(g.standard_normal((R, V)) * scale).to(dtype).cuda()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("R,V,n_top", [
    (1, 1, 1), (2, 2, 5), (3, 7, 32), (5, 64, 8), (1, 255, 20), (4, 1000, 32), (2, 1024, 1), (7, 1025, 4), (40, 8191, 20), (3, 16384, 32),
    (1, 50257, 20), (2, 129283, 32), (64, 32769, 8), (330, 4099, 3), (9, 131072, 0), (1, 1 << 20, 32),
])
def test_logprobs(R, V, n_top, dtype):
    g = np.random.default_rng(R + V + n_top)
    tokens = g.integers(-1, V, (R, 3)).astype(np.int32)
    check(draw(g, R, V, dtype), tokens, 1.0 if V % 2 else 0.7, n_top)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("off,pad", [(0, 1), (1, 0), (3, 5), (7, 64), (5, 2)])
def test_rows_of_a_wider_array(dtype, off, pad):
    """Rows that start anywhere; what lies around them (NaN here) is not used."""
    g = np.random.default_rng(off + pad)
    full = torch.full((6, off + 3001 + pad), float("nan"), dtype=dtype, device="cuda")
    full[:, off:off + 3001] = draw(g, 6, 3001, dtype)
    check(full[:, off:off + 3001], g.integers(0, 3001, (6, 2)).astype(np.int32), 1.25, 9)


@pytest.mark.parametrize("V", [300, 20000, 140000])
@pytest.mark.parametrize("R", [3, 200])
def test_ties_and_masks(R, V):
    g = np.random.default_rng(V + R)
    x = torch.from_numpy(g.integers(-3, 4, (R, V)).astype(np.float32)).cuda()
    x[0] = 0.0                                # one value, both zeros
    x[0, ::3] = -0.0
    x[1] = -INF                               # every token ruled out
    x[2] = -INF
    x[2, [V - 1, V // 2, 5]] = torch.tensor([1.0, 1.0, -2.0], device="cuda")
    if R > 10:
        x[3] = torch.arange(V, device="cuda") / V            # ascending
        x[4] = -torch.arange(V, device="cuda") / V
        x[5] = torch.finfo(torch.float32).min                # masks of the type's lowest value: all, and all but one
        x[6] = torch.finfo(torch.bfloat16).min
        x[6, V - 2] = 3.0
        x[7, V // 3:] = -INF
        x[8] *= 1000.0                                       # one token has it all
        x[9] = 1e30
    for dtype in (torch.float32, torch.bfloat16):
        check(x.to(dtype), g.integers(0, V, (R, 4)).astype(np.int32), 1.0, 32)


def test_tokens_out_of_range_and_parts():
    c.csa2_device_flags()
    g = np.random.default_rng(8)
    x = draw(g, 4, 100, torch.float32)
    tokens = np.array([[-1, 100], [5, -7], [1 << 30, 0], [99, 99]], np.int32)
    lp, lse, ent, ti, tl = check(x, tokens, 1.0, 6)
    assert c.csa2_device_flags() == c.FLAG_INDEX_OOB
    # any part alone gives the same
    one = torch.zeros_like(ti)
    c.csa2_token_logprobs(x, top_ids=one)
    assert torch.equal(one, ti)
    one = torch.zeros_like(lse)
    c.csa2_token_logprobs(x, lse=one)
    assert torch.equal(one, lse)
    one = torch.zeros_like(tl)
    c.csa2_token_logprobs(x, top_logprobs=one)
    assert torch.equal(one, tl)


def test_captured_on_a_stream():
    g = np.random.default_rng(9)
    x = draw(g, 5, 30000, torch.bfloat16)
    tokens = to_dev(g.integers(0, 30000, (5, 1)).astype(np.int32))
    lp, ids = torch.zeros((5, 1), device="cuda"), torch.zeros((5, 4), dtype=torch.int32, device="cuda")
    call = lambda: c.csa2_token_logprobs(x, tokens, lp, top_ids=ids)  # noqa: E731
    call()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for seed in (1, 2):
        x.copy_(draw(np.random.default_rng(seed), 5, 30000, torch.bfloat16))
        graph.replay()
        got = lp.clone(), ids.clone()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        c.csa2_token_logprobs(x, tokens, lp, top_ids=ids, stream=side)
        side.synchronize()
        assert torch.equal(got[0], lp) and torch.equal(got[1], ids)


def test_offsets_past_32_bits():
    """Rows of a logits array of more than 2^32 bytes: the last ones are read where they lie."""
    V, R = 131072, 16400
    x = torch.zeros((R, V), dtype=torch.bfloat16, device="cuda")
    g = np.random.default_rng(10)
    x[-3:] = draw(g, 3, V, torch.bfloat16)
    ids, lse = torch.zeros((R, 2), dtype=torch.int32, device="cuda"), torch.zeros((R,), device="cuda")
    c.csa2_token_logprobs(x, lse=lse, top_ids=ids)
    assert torch.equal(ids[:-3].cpu(), torch.tensor([[0, 1]], dtype=torch.int32).expand(R - 3, 2))
    assert torch.allclose(lse[:-3], torch.full((R - 3,), float(np.log(V)), device="cuda"), atol=1e-5, rtol=0)
    want = P.logprobs(host(x[-3:]), np.zeros((3, 1), np.int32), 1.0, 2)
    assert np.array_equal(host(ids[-3:]), want[3])


@pytest.mark.parametrize("R,V", [(700, 20000), (330, 66001), (1300, 5200)])
def test_ties_and_masks_of_many_rows(R, V):
    test_ties_and_masks(R, V)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("R", [3, 400])
@pytest.mark.parametrize("n_top", [1, 5, 32])
def test_candidates_of_few_and_many_lanes(R, n_top, dtype):
    """The likeliest tokens one, four, five or all 32 to a group, in one lane or in several, and more of them than count."""
    V = 30011
    g = np.random.default_rng(R + n_top)
    x = draw(g, R, V, dtype).clamp(max=3.0)
    for i in range(R):
        start = int(g.integers(0, V - 300))
        step = (1, 8, 9, 3)[i % 4]
        count = (1, 4, 5, 33)[i // 4 % 4]
        at = start + step * np.arange(count)
        values = 50.0 + (0.5 * (np.arange(count) % 3) if i % 2 else np.zeros(count))
        x[i, torch.from_numpy(at).cuda()] = torch.from_numpy(values).to(dtype).cuda()
    check(x, g.integers(0, V, (R, 2)).astype(np.int32), 1.0, n_top)
