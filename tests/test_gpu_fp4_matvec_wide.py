"""Products over more channels than 32-bit sizes of x hold."""
import numpy as np
import pytest

from tests import _verify as V
from tests._cases import to_dev

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)
import compressed_sparse_attention_step_gb300 as c  # noqa: E402


def test_two_to_the_27_channels():
    """17 token rows of which 512 channels from end to end are not zero: y is the sum over these alone.  The bound
    is that of 512 products: 8 accumulations a block, a sum over the 48 blocks that hold them, and 80 of warps and
    clusters, 2^-22 each."""
    M, N, K = 17, 32, 1 << 27
    g = np.random.default_rng(5)
    codes = torch.zeros((N, K // 2), dtype=torch.uint8, device="cuda")
    scales = torch.full((N, K // 16), 0x7E, dtype=torch.uint8, device="cuda")
    x = torch.zeros((M, K), dtype=torch.bfloat16, device="cuda")
    at = np.sort(np.concatenate((np.arange(128), np.arange(K - 128, K), g.choice(K // 256 - 2, 16, replace=False)
                                 .repeat(16) * 256 + 256 + np.tile(np.arange(16), 16))))
    wc, ws = V.random_fp4(g, N, 512)
    w = V.dequant(wc, ws)
    groups = at[::16] // 16
    assert (at.reshape(-1, 16) // 16 == groups[:, None]).all()
    for i, gr in enumerate(groups):
        codes[:, 8 * gr:8 * gr + 8] = to_dev(np.ascontiguousarray(wc[:, 8 * i:8 * i + 8]))
        scales[:, gr] = to_dev(np.ascontiguousarray(ws[:, i]))
    xs = torch.randn((M, 512), generator=torch.Generator().manual_seed(3)).bfloat16()
    x[:, torch.from_numpy(at).cuda()] = xs.cuda()
    packed = c.fp4_weight_alloc(N, K)
    c.csa2_fp4_pack_weight(codes, scales, packed)
    del codes, scales
    y = torch.full((M, N), 7.0, dtype=torch.float32, device="cuda")
    c.csa2_device_flags()
    c.csa2_fp4_matvec(x, packed, y)
    assert c.csa2_device_flags() == 0
    xd = xs.double().numpy()
    err = np.abs(y.cpu().numpy() - xd @ w.T)
    assert (err <= (np.abs(xd) @ np.abs(w).T) * (8 + 48 + 80) * 2.0 ** -22).all()
