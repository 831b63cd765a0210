"""Low-rank adapters of many requests against a plain 64-bit form."""
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


def host(t):
    return t.float().cpu().numpy().astype(np.float64)


def make(seed, m, n_in, n_out, r, L, fp32, order="mixed", none=0.2):
    g = np.random.default_rng(seed)
    if order == "runs":
        adapter = np.repeat(g.integers(-1, L, m), g.integers(1, 90, m))[:m].astype(np.int32)
    else:
        adapter = np.where(g.random(m) < none, -1, g.integers(0, max(L, 1), m) if L else -1).astype(np.int32)
    x, a, b = V.bf16(g, (m, n_in)), V.bf16(g, (L, r, n_in), max(n_in, 1) ** -0.5), V.bf16(g, (L, n_out, r))
    base = torch.from_numpy(g.standard_normal((m, n_out))).to(torch.float32 if fp32 else torch.bfloat16).cuda()
    return g, adapter, x, a, b, base


@pytest.mark.parametrize("m,n_in,n_out,r,L", [
    (1, 8, 1, 8, 1), (1, 4096, 4096, 16, 3), (3, 40, 33, 8, 2), (16, 256, 264, 16, 16), (17, 136, 100, 24, 5), (64, 512, 200, 32, 64),
    (33, 1000, 72, 64, 4), (40, 64, 31, 128, 3), (100, 328, 40, 40, 7), (511, 96, 50, 8, 2), (512, 96, 56, 16, 3), (700, 256, 333, 64, 9),
    (1100, 72, 96, 128, 2), (600, 2056, 24, 32, 40), (5, 0, 9, 8, 2), (7, 16, 9, 8, 0),
])
@pytest.mark.parametrize("fp32", [False, True])
@pytest.mark.parametrize("order", ["mixed", "runs"])
def test_adapters(m, n_in, n_out, r, L, fp32, order):
    g, adapter, x, a, b, base = make(m + n_in + r, m, n_in, n_out, r, L, fp32, order)
    ranks = g.integers(0, r + 1, L).astype(np.int32) if m % 2 else None
    scale = (g.random(L) * 3 - 1).astype(np.float32) if m % 3 else None
    ad, bd = bf16_dev(a), bf16_dev(b)
    if ranks is not None:   # what lies past a rank is not used
        for l in range(L):
            ad[l, int(ranks[l]):] = float("nan")
            bd[l, :, int(ranks[l]):] = float("nan")
    out = torch.full_like(base, 9.0)
    args = (bf16_dev(x), ad, bd, to_dev(adapter), base)
    kw = dict(ranks=None if ranks is None else to_dev(ranks), scale=None if scale is None else to_dev(scale))
    c.csa2_lora_add(*args, out, **kw)
    exact, tol = P.adapters(V.f64(x), V.f64(a), V.f64(b), adapter, host(base), ranks, scale,
                            split=2.0 ** -24 if fp32 else 2.0 ** -16)   # fp32: three terms
    err = np.abs(host(out) - exact)
    tol = P.rounded(exact, tol, not fp32)
    assert (err <= tol).all(), f"{np.max(err - tol):.3e} over the bound"
    none = adapter < 0
    assert torch.equal(out[to_dev(none)], base[to_dev(none)])
    c.csa2_lora_add(*args, base, **kw)   # in place
    assert torch.equal(out, base)


def test_other_rows_do_not_matter():
    """Rows of other adapters in a tile, infinities and NaN among them, change nothing."""
    g, adapter, x, a, b, base = make(1, 48, 160, 80, 16, 4, True, none=0.0)
    adapter[:] = np.arange(48) % 4
    outs = []
    for other in (0.0, float("inf"), float("nan")):
        xd, out = bf16_dev(x), torch.zeros_like(base)
        xd[to_dev(adapter != 2)] = other
        c.csa2_lora_add(xd, bf16_dev(a), bf16_dev(b), to_dev(adapter), base, out)
        outs.append(out[to_dev(adapter == 2)])
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])


def test_adapters_out_of_range_are_none():
    c.csa2_device_flags()
    g, adapter, x, a, b, base = make(2, 20, 64, 40, 8, 3, False)
    adapter[[2, 11]] = 3, 1 << 30
    adapter[5] = -(1 << 31)
    out = torch.zeros_like(base)
    c.csa2_lora_add(bf16_dev(x), bf16_dev(a), bf16_dev(b), to_dev(adapter), base, out)
    assert torch.equal(out[[2, 5, 11]], base[[2, 5, 11]])
    assert c.csa2_device_flags() == c.FLAG_INDEX_OOB


@pytest.mark.parametrize("m", [40, 640])
def test_captured(m):
    g, adapter, x, a, b, base = make(3, m, 256, 520, 32, 6, False)
    xd, ad, bd, out = bf16_dev(x), bf16_dev(a), bf16_dev(b), torch.zeros_like(base)
    which = to_dev(adapter)
    call = lambda: c.csa2_lora_add(xd, ad, bd, which, base, out)  # noqa: E731
    call()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
        call()
    for seed in (4, 5):
        _, adapter, x, _, _, _ = make(seed, m, 256, 520, 32, 6, False)
        xd.copy_(bf16_dev(x))
        which.copy_(to_dev(adapter))
        graph.replay()
        exact, tol = P.adapters(V.f64(x), V.f64(a), V.f64(b), adapter, host(base))
        assert (np.abs(host(out) - exact) <= P.rounded(exact, tol, True)).all()


# Many rows of few adapters: tiles of 64 rows, over the end of a window of 8192 too
TALL = [(5600, 520, 512, 16, 5), (5000, 1000, 333, 64, 8), (9000, 264, 776, 32, 3), (6000, 512, 520, 128, 6), (8192, 600, 500, 40, 1),
        (6100, 1024, 264, 8, 7), (16500, 328, 712, 64, 4), (4900, 2056, 72, 24, 2)]


@pytest.mark.parametrize("m,n_in,n_out,r,L", TALL)
@pytest.mark.parametrize("fp32", [False, True])
@pytest.mark.parametrize("order", ["mixed", "runs"])
def test_tall_tiles(m, n_in, n_out, r, L, fp32, order):
    test_adapters(m, n_in, n_out, r, L, fp32, order)


def test_tall_tiles_other_rows_do_not_matter():
    g, adapter, x, a, b, base = make(1, 6000, 512, 520, 64, 4, True, none=0.0)
    adapter[:] = np.arange(6000) % 4
    outs = []
    for other in (0.0, float("inf"), float("nan")):
        xd, out = bf16_dev(x), torch.zeros_like(base)
        xd[to_dev(adapter != 2)] = other
        c.csa2_lora_add(xd, bf16_dev(a), bf16_dev(b), to_dev(adapter), base, out)
        outs.append(out[to_dev(adapter == 2)])
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])


def test_rows_of_a_shared_bucket():
    """Adapters whose numbers are equal modulo 255 meet in tiles, tall ones among them."""
    for m in (50, 8192):
        L = 700
        g, adapter, x, a, b, base = make(6, m, 72, 1032, 40, L, False)
        adapter[:] = np.where(adapter < 0, -1, adapter % 3 * 255 + g.integers(0, 2, m))
        out = torch.zeros_like(base)
        c.csa2_lora_add(bf16_dev(x), bf16_dev(a), bf16_dev(b), to_dev(adapter), base, out)
        exact, tol = P.adapters(V.f64(x), V.f64(a), V.f64(b), adapter, host(base))
        assert (np.abs(host(out) - exact) <= P.rounded(exact, tol, True)).all()


@pytest.mark.parametrize("none", [0.0, 0.03, 0.97, 1.0])
@pytest.mark.parametrize("m", [70, 5000])
def test_rows_without_an_adapter(m, none):
    g, adapter, x, a, b, base = make(7, m, 512, 520, 32, 3, False, none=none)
    out = torch.full_like(base, 9.0)
    c.csa2_lora_add(bf16_dev(x), bf16_dev(a), bf16_dev(b), to_dev(adapter), base, out)
    exact, tol = P.adapters(V.f64(x), V.f64(a), V.f64(b), adapter, host(base))
    assert (np.abs(host(out) - exact) <= P.rounded(exact, tol, True)).all()
    off = to_dev(adapter < 0)
    assert torch.equal(out[off], base[off])
