"""The block-scaled product over its tiles: sizes that the choice gives to
each (256x256, 256x128, 128x128, 128x64, 64x64), split and not, with every
remainder of k-blocks against the loops' unrolling, ends inside tiles and
blocks, in all pairs of formats. Reference: 64-bit products of the stored
values, which bf16 holds exactly here."""
import pytest
import torch

import tensor_scaled_fp8_amd as tsf
from tests.block_util import BF16_HALF, MFMA

pytestmark = pytest.mark.gpu


def _stored(g, rows, cols, fmt):
    x = torch.randn((rows, cols), generator=g, device="cuda")
    # scales that differ from row to row and from block to block
    x *= torch.exp2(torch.randint(-4, 5, (rows, 1), generator=g, device="cuda").float())
    nb = -(-cols // 128)
    x *= torch.exp2(torch.randint(-4, 5, (1, nb), generator=g, device="cuda").float()).repeat_interleave(128, 1)[:, :cols]
    q = tsf.fp8_block_quantize(x.to(torch.bfloat16), fmt)[0]
    return q, q.dequantize().double()


SIZES = [(4000, 4100, 390), (4096, 4096, 500), (3900, 4000, 640), (1000, 8000, 640), (2000, 2100, 1200),
         (4000, 4100, 1300), (1800, 4000, 3000), (1000, 8000, 130), (2048, 2048, 300), (1900, 2001, 900),
         (1500, 6000, 700), (3000, 3001, 1400), (1024, 2048, 700), (997, 2002, 1200), (1000, 2000, 1025),
         (4100, 4100, 3000), (2300, 8000, 2500), (333, 2222, 1111), (60, 500, 6000), (513, 1030, 4000), (1100, 1100, 10000), (1500, 3000, 6000),
         (2048, 4096, 20480)]


@pytest.mark.parametrize("at", range(len(SIZES)))
def test_tiles(at):
    M, N, R = SIZES[at]
    fa, fb = (("e4m3", "e4m3"), ("e5m2", "e4m3"), ("e4m3", "e5m2"), ("e5m2", "e5m2"))[at % 4]
    g = torch.Generator("cuda").manual_seed(at)
    a, va = _stored(g, M, R, fa)
    b, vb = _stored(g, N, R, fb)
    wide = torch.full((M, N + 5), 3.0, dtype=torch.bfloat16, device="cuda")
    out = tsf.fp8_block_gemm(a, b, wide[:, :N])
    want = torch.matmul(va, vb.t().contiguous())
    tol = BF16_HALF * want.abs() + MFMA * torch.matmul(va.abs(), vb.abs().t().contiguous())
    bad = ~((out.double() - want).abs() <= tol)
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[0].tolist())
    assert (wide[:, N:] == 3.0).all()
    for _ in range(3):
        assert torch.equal(tsf.fp8_block_gemm(a, b), out)          # the same bits every time


def test_no_second_backward_through_the_first():
    """The gradients are made by kernels: a graph of them is refused, not taken for a constant."""
    G = torch.randn((3, 128), device="cuda").to(torch.bfloat16).requires_grad_()
    W = torch.randn((128, 4), device="cuda").to(torch.bfloat16).requires_grad_()
    for y in (tsf.swiglu(G, G), tsf.block_linear(G, W)):
        d, = torch.autograd.grad(y, G, torch.ones_like(y).requires_grad_(), create_graph=True)
        with pytest.raises(RuntimeError):
            d.float().sum().backward()
