"""The serving linear at the sizes where its form changes: fused and stored
X, one or two 16-row fragments, 1 to 3 column blocks a workgroup, k-blocks
that do not divide among the waves, ends inside a block, odd pitches."""
import numpy as np
import pytest
import torch

import tensor_scaled_fp8_amd as tsf
from tests.block_util import BF16_HALF, MFMA, held, to_bf16

pytestmark = pytest.mark.gpu


def _up(x):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).cuda().to(torch.bfloat16)


def _check(x, w, y):
    a, b = held(x), held(w.T)
    want = a @ b.T
    got = y.float().cpu().numpy().astype(np.float64)
    assert got.shape == want.shape
    bad = ~(np.abs(got - want) <= BF16_HALF * np.abs(want) + MFMA * (np.abs(a) @ np.abs(b).T) + 2.0 ** -133)
    assert not bad.any(), (bad.sum(), np.argwhere(bad)[0])


@pytest.mark.parametrize("M,K,N", [(1, 128, 16), (1, 1, 1), (1, 7, 300), (2, 8, 5), (1, 1111, 777), (3, 2048, 130),
                                   (4, 5000, 33), (16, 2048, 64), (16, 2050, 64), (7, 4700, 257), (13, 700, 4500),
                                   (1, 640, 9000), (16, 2200, 9001), (11, 3000, 13000), (17, 130, 4096),
                                   (31, 1100, 4100), (32, 900, 8500), (20, 520, 500), (33, 500, 4200)])
def test_serve_forms(M, K, N):
    g = np.random.Generator(np.random.PCG64(M * K + N))
    x = to_bf16(g.standard_normal((M, K)) * np.exp2(g.integers(-6, 6, size=(M, 1))))
    w = to_bf16(g.standard_normal((K, N)) * np.exp2(g.integers(-4, 4, size=(1, N))) * 0.02)
    wide = torch.full((M, K + 3), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[:, 1:K + 1] = _up(x)
    w8 = tsf.prepare_block_weight(_up(w))
    y = tsf.fp8_block_linear_fwd_cached(wide[:, 1:K + 1], w8)
    _check(x, w, y)
    assert torch.equal(tsf.fp8_block_linear_fwd_cached(_up(x), w8), y)      # any pitch, the same bits


def test_serve_scratch_form_gives_the_same_bits():
    """The entry point with scratch, at sizes of the form that takes none."""
    g = np.random.Generator(np.random.PCG64(5))
    M, K, N = 3, 1500, 400
    x, w = _up(g.standard_normal((M, K))), _up(g.standard_normal((K, N)))
    w8 = tsf.prepare_block_weight(w)
    want = tsf.fp8_block_linear_fwd_cached(x, w8)
    lib = tsf.load()
    assert lib.fp8_block_linear_few(M, K, N) == 1
    nb = lib.fp8_block_linear_cached_bytes(M, K, N)
    ws = torch.empty(nb, dtype=torch.uint8, device="cuda")
    y = torch.empty((M, N), dtype=torch.bfloat16, device="cuda")
    c, s = w8.pointers()
    assert lib.fp8_block_linear_fwd_cached(x.data_ptr(), K, M, K, N, c, s, ws.data_ptr(), nb, y.data_ptr(),
                                           torch.cuda.current_stream().cuda_stream) == 0
    assert torch.equal(y, want)


@pytest.mark.parametrize("M", [1, 20])
def test_serve_nonfinite(M):
    """A NaN stays in its row; an infinity saturates its block."""
    g = np.random.Generator(np.random.PCG64(6))
    K, N = 700, 4100
    x, w = to_bf16(g.standard_normal((M, K))), to_bf16(g.standard_normal((K, N)))
    x[M - 1, 5] = np.inf
    y = tsf.fp8_block_linear_fwd_cached(_up(x), tsf.prepare_block_weight(_up(w)))
    _check(x, w, y)
    x[0, 699] = np.nan
    y = tsf.fp8_block_linear_fwd_cached(_up(x), tsf.prepare_block_weight(_up(w)))
    nan = torch.zeros((M, N), dtype=torch.bool, device="cuda")
    nan[0] = True
    assert torch.equal(torch.isnan(y), nan)


def test_serve_in_a_graph():
    g = np.random.Generator(np.random.PCG64(7))
    K, N = 900, 600
    w8 = tsf.prepare_block_weight(_up(g.standard_normal((K, N))))
    x = _up(g.standard_normal((2, K)))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        tsf.fp8_block_linear_fwd_cached(x, w8)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = tsf.fp8_block_linear_fwd_cached(x, w8)
    for _ in range(3):
        new = _up(g.standard_normal((2, K)))
        want = tsf.fp8_block_linear_fwd_cached(new, w8)
        x.copy_(new)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want)
