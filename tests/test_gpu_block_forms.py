"""The block-scaled product in the forms that the sizes of
test_gpu_block_tiles.py leave out: split 256x128 and 128x64 tiles and the
remaining numbers of k-blocks modulo the loops' unrolling, each in all pairs of
formats. test_block_forms_host.py asserts that the two lists together reach
every form. Reference: 64-bit products of the stored values."""
import pytest
import torch

import tensor_scaled_fp8_amd as tsf
from tests.block_util import BF16_HALF, MFMA
from tests.test_gpu_block_tiles import _stored

pytestmark = pytest.mark.gpu

SIZES = [(69, 35, 139), (35, 40, 263), (775, 1219, 260), (1602, 577, 386), (452, 323, 4655), (1161, 1686, 513),
         (2315, 1683, 771), (1032, 3593, 902), (1411, 2713, 1026), (647, 2695, 6409), (2333, 3353, 771),
         (1668, 4674, 259)]


@pytest.mark.parametrize("fa,fb", [("e4m3", "e4m3"), ("e5m2", "e4m3"), ("e4m3", "e5m2"), ("e5m2", "e5m2")])
@pytest.mark.parametrize("M,N,R", SIZES)
def test_forms(M, N, R, fa, fb):
    g = torch.Generator("cuda").manual_seed(M + N + R)
    a, va = _stored(g, M, R, fa)
    b, vb = _stored(g, N, R, fb)
    wide = torch.full((M, N + 3), 3.0, dtype=torch.bfloat16, device="cuda")
    out = tsf.fp8_block_gemm(a, b, wide[:, :N])
    want = torch.matmul(va, vb.t().contiguous())
    tol = BF16_HALF * want.abs() + MFMA * torch.matmul(va.abs(), vb.abs().t().contiguous())
    bad = ~((out.double() - want).abs() <= tol)
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[0].tolist())
    assert (wide[:, N:] == 3.0).all()
    assert torch.equal(tsf.fp8_block_gemm(a, b), out)              # the same bits every time
