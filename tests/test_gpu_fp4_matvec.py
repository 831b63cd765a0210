"""Products of token rows with a packed 4-bit weight against a plain 64-bit form, bound by bound."""
import numpy as np
import pytest

import csa2_synth as syn
from tests import _verify as V
from tests._cases import bf16_dev, to_dev

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)
import compressed_sparse_attention_step_gb300 as c  # noqa: E402


def _weight(g, N, K, lo=0x20, hi=0x50):
    codes, scales = V.random_fp4(g, N, K, lo, hi)
    packed = c.fp4_weight_alloc(N, K)
    c.csa2_fp4_pack_weight(to_dev(codes), to_dev(scales), packed)
    return packed, V.dequant(codes, scales)


def _check(y, x, w, rs, what=""):
    """|y - exact| <= sum |x w| times 2^-22 for each accumulation of the longest path (a block's 8, its scaling
    and sum over the blocks, the warps' and the cluster's sums), 2^-38 of a block's largest |x| for an x below
    f16's range, the product with row_scale, and the rounding to bf16."""
    M, K = x.shape
    exact = (x @ w.T) * rs
    mag = (np.abs(x) @ np.abs(w).T) * np.abs(rs)
    n_kb = -(-K // 128)
    pad = np.pad(np.abs(x), ((0, 0), (0, n_kb * 128 - K))).reshape(M, n_kb, 128)
    big = np.repeat(pad.max(-1, keepdims=True), 128, -1).reshape(M, -1)[:, :K]
    tol = mag * (8 + n_kb + 80) * 2.0 ** -22 + (big @ np.abs(w).T) * np.abs(rs) * 2.0 ** -38 + np.abs(exact) * 2.0 ** -22
    if y.dtype == torch.bfloat16:
        tol = tol + np.abs(exact) * 2.0 ** -8
    err = np.abs(y.float().cpu().numpy().astype(np.float64) - exact)
    assert (err <= tol + 1e-38).all(), f"{what}: {np.max(err - tol):.3e} over the bound"


@pytest.mark.parametrize("M,N,K", [
    (1, 1, 16), (1, 4, 128), (2, 16, 128), (3, 17, 144), (8, 33, 112), (9, 100, 1040), (16, 64, 2048), (17, 40, 400),
    (24, 31, 272), (25, 512, 512), (32, 300, 640), (32, 5, 48), (1, 512, 4096), (5, 1000, 1056), (7, 5000, 256),
    (32, 5120, 384), (12, 20000, 48), (4, 16, 33008), (32, 16, 20000), (1, 40000, 32), (20, 9000, 160),
    # the tensor-memory form: odd rows and channels, one and two channel blocks per CTA, shares of more than 2048
    # channels, ten token rows; and an x that no cluster holds
    (17, 2080, 4112), (24, 16500, 512), (20, 9001, 1024), (32, 1030, 8176), (18, 4100, 2320), (12, 8200, 8208),
    (32, 1000, 33008),
    # clusters of eight, and two passes of 16 rows
    (32, 1200, 12304), (16, 4200, 17008), (24, 1031, 16400), (17, 300, 32768),
])
@pytest.mark.parametrize("fp32", [False, True])
def test_matvec(M, N, K, fp32):
    g = np.random.default_rng(M * 7 + N + K)
    packed, w = _weight(g, N, K)
    xb = V.bf16(g, (M, K))
    rs = (g.random(N) * 2 - 0.5).astype(np.float32)
    y = torch.full((M, N), 7.0, dtype=torch.float32 if fp32 else torch.bfloat16, device="cuda")
    c.csa2_fp4_matvec(bf16_dev(xb), packed, y, row_scale=to_dev(rs))
    _check(y, V.f64(xb), w, rs.astype(np.float64))
    first = y.clone()
    c.csa2_fp4_matvec(bf16_dev(xb), packed, y, row_scale=to_dev(rs))
    assert torch.equal(first, y)


def test_every_code_and_scale():
    """One-hot tokens read single weights back: every code, and every finite scale byte, exactly."""
    scales = np.array([b for b in range(256) if b & 0x7F != 0x7F], np.uint8)
    N = len(scales)
    codes = np.tile(np.array([2 * i + ((2 * i + 1) << 4) for i in range(8)], np.uint8), (N, 1))      # K = 16
    packed = c.fp4_weight_alloc(N, 16)
    c.csa2_fp4_pack_weight(to_dev(codes), to_dev(scales[:, None]), packed)
    y = torch.empty((16, N), dtype=torch.float32, device="cuda")
    c.csa2_fp4_matvec(bf16_dev(syn.f32_to_bf16_bits(np.eye(16, dtype=np.float32))), packed, y)
    # (16 tokens: y[m][n] = weight n, channel m)
    assert np.array_equal(y.cpu().numpy().astype(np.float64), V.dequant(codes, scales[:, None]).T)


@pytest.mark.parametrize("scale", [2.0 ** -120, 2.0 ** -60, 2.0 ** 60, 2.0 ** 100])
def test_x_of_any_magnitude(scale):
    """Each token's blocks are scaled into f16's range on their own: tiny, huge and mixed ones."""
    g = np.random.default_rng(3)
    packed, w = _weight(g, 70, 512)
    x = g.standard_normal((6, 512)) * scale
    x[1] = 0
    x[2, :128] *= 2.0 ** -20
    x[3, 7] *= 2.0 ** 20
    xb = syn.f32_to_bf16_bits(x.astype(np.float32))
    y = torch.empty((6, 70), dtype=torch.float32, device="cuda")
    c.csa2_fp4_matvec(bf16_dev(xb), packed, y)
    _check(y, V.f64(xb), w, np.ones(70))
    assert (y[1] == 0).all()


def test_a_token_with_infinities_spoils_no_other():
    g = np.random.default_rng(4)
    packed, w = _weight(g, 40, 256)
    xb = V.bf16(g, (3, 256))
    xb[1, 5] = 0x7F80
    y = torch.empty((3, 40), dtype=torch.bfloat16, device="cuda")
    c.csa2_fp4_matvec(bf16_dev(xb), packed, y)
    keep = [0, 2]
    _check(y[keep], V.f64(xb[keep]), w, np.ones(40))


def test_rows_of_the_cache_are_weights(orc):
    """A cache's FP4 rows (csa2_fp4_quantize_append) are a weight of 512 input channels."""
    x = syn.outlier_bf16(1, syn.T_X, 0, (48, 512))
    codes = torch.empty((1, 48, 256), dtype=torch.uint8, device="cuda")
    scales = torch.empty((1, 48, 32), dtype=torch.uint8, device="cuda")
    c.csa2_fp4_quantize_append(bf16_dev(x)[None], codes, scales)
    packed = c.fp4_weight_alloc(48, 512)
    c.csa2_fp4_pack_weight(codes[0], scales[0], packed)
    w = V.f64(orc.fp4_dequantize(*orc.fp4_quantize(x)))
    g = np.random.default_rng(2)
    xb = V.bf16(g, (2, 512))
    y = torch.empty((2, 48), dtype=torch.float32, device="cuda")
    c.csa2_fp4_matvec(bf16_dev(xb), packed, y)
    _check(y, V.f64(xb), w, np.ones(48))


def test_captured_and_on_another_stream():
    g = np.random.default_rng(9)
    packed, w = _weight(g, 600, 1024)
    xb = V.bf16(g, (11, 1024))
    x = bf16_dev(xb)
    y = torch.empty((11, 600), dtype=torch.float32, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        c.csa2_fp4_matvec(x, packed, y)
    s.synchronize()
    _check(y, V.f64(xb), w, np.ones(600))
    ref = y.clone()
    graphs = []
    for _ in range(2):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            c.csa2_fp4_matvec(x, packed, y)
        graphs.append(gr)
    y.zero_()
    for gr in graphs:
        gr.replay()
    torch.cuda.synchronize()
    assert torch.equal(ref, y)


def test_two_calls_at_once():
    """Two streams, both kernels, different inputs."""
    g = np.random.default_rng(10)
    jobs = []
    for M, N, K in ((20, 2300, 4096), (3, 700, 640), (32, 4096, 2100 // 16 * 16)):
        packed, w = _weight(g, N, K)
        xb = V.bf16(g, (M, K))
        jobs.append((bf16_dev(xb), packed, torch.empty((M, N), dtype=torch.float32, device="cuda"), xb, w,
                     torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(20):
        for x, packed, y, _, _, s in jobs:
            c.csa2_fp4_matvec(x, packed, y, stream=s)
    torch.cuda.synchronize()
    for x, packed, y, xb, w, _ in jobs:
        _check(y, V.f64(xb), w, np.ones(y.shape[1]))
    assert c.csa2_device_flags() == 0


@pytest.mark.parametrize("M,N,K", [(19, 28, 6240), (9, 35, 3568), (20, 9, 3792), (5, 64, 2048), (12, 100, 1040),
                                   (32, 512, 4096), (16, 300, 8192), (24, 4100, 4112),
                                   # many blocks a warp: slots of its ring are refilled behind their reads
                                   (32, 1030, 8176), (32, 2048, 8192), (8, 1030, 16384), (2, 40, 32768)])
def test_calls_behind_one_another(M, N, K):
    """Clusters that exchange partial sums, call upon call with nothing between: each gives the first one's bits."""
    g = np.random.default_rng(M + N)
    packed, w = _weight(g, N, K)
    xb = V.bf16(g, (M, K))
    x = bf16_dev(xb)
    buf = torch.full((100, -(-M * N // 4) * 4), 7.0, dtype=torch.float32, device="cuda")      # each starts on 16 bytes
    ys = [b[:M * N].view(M, N) for b in buf]
    for y in ys:
        c.csa2_fp4_matvec(x, packed, y)
    _check(ys[0], V.f64(xb), w, np.ones(N))
    assert torch.equal(buf, buf[:1].expand_as(buf))


@pytest.mark.parametrize("M", [2, 32])
def test_a_weight_of_more_than_4_gb(M):
    """The last rows of a weight whose blocks lie past 32 bits; all others are zero."""
    N, K, last = 1_000_100, 8192, 70
    g = np.random.default_rng(M)
    codes, scales = V.random_fp4(g, last, K)
    dc, ds = torch.zeros((N, K // 2), dtype=torch.uint8, device="cuda"), torch.zeros((N, K // 16), dtype=torch.uint8, device="cuda")
    dc[-last:], ds[-last:] = to_dev(codes), to_dev(scales)
    packed = c.fp4_weight_alloc(N, K)
    assert packed.numel() > 2 ** 32
    c.csa2_fp4_pack_weight(dc, ds, packed)
    xb = V.bf16(g, (M, K))
    y = torch.full((M, N), 7.0, dtype=torch.float32, device="cuda")
    c.csa2_fp4_matvec(bf16_dev(xb), packed, y)
    _check(y[:, -last:], V.f64(xb), V.dequant(codes, scales), np.ones(last))
    assert bool((y[:, :-last] == 0).all())


@pytest.mark.parametrize("M,N,K", [
    # on both sides of where the tensor-memory form begins: rows, channels and weight
    (32, 4097, 2048), (25, 4100, 1920), (25, 5000, 2064), (24, 2080, 4096), (24, 4200, 3968), (17, 2016, 4096),
    (16, 8200, 8192), (16, 16400, 8064), (9, 8170, 8192), (9, 10000, 8208), (8, 8200, 8192), (16, 33000, 4096),
])
def test_matvec_at_the_forms_borders(M, N, K):
    g = np.random.default_rng(M + N + K)
    packed, w = _weight(g, N, K)
    xb = V.bf16(g, (M, K))
    rs = (g.random(N) * 2 - 0.5).astype(np.float32)
    y = torch.full((M, N), 7.0, dtype=torch.float32, device="cuda")
    c.csa2_device_flags()
    c.csa2_fp4_matvec(bf16_dev(xb), packed, y, row_scale=to_dev(rs))
    assert c.csa2_device_flags() == 0
    _check(y, V.f64(xb), w, rs.astype(np.float64))
