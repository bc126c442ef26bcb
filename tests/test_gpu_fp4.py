"""4-bit weights: stored and restored exactly, and the linear on them against
the definition in 64 bits."""
import numpy as np
import pytest
import torch

import tensor_scaled_fp8_amd as tsf
from tests.block_util import BF16_HALF, MFMA, held, to_bf16
from tests.serve_util import GRID, fp4_held

pytestmark = pytest.mark.gpu


def up(x):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).cuda().to(torch.bfloat16)


def host(t):
    return t.float().cpu().numpy().astype(np.float64)


def weight(g, K, N):
    return to_bf16(g.standard_normal((K, N)) * np.exp2(g.integers(-4, 4, size=(1, N))) * 0.02)


@pytest.mark.parametrize("K,N", [(1, 1), (32, 16), (33, 17), (511, 40), (512, 3), (700, 65), (96, 300)])
def test_store_and_restore(K, N):
    g = np.random.Generator(np.random.PCG64(K + N))
    w = weight(g, K, N)
    wide = torch.zeros((K, N + 3), dtype=torch.bfloat16, device="cuda")
    wide[:, 1:N + 1] = up(w)
    q = tsf.prepare_fp4_weight(wide[:, 1:N + 1])
    assert q.shape == (K, N) and q.nbytes == -(-N // 16) * -(-K // 512) * 4 * 1088
    assert np.array_equal(host(q.dequantize()), fp4_held(w))


def test_borders_and_extremes():
    """Every value, the middles between them and their neighbours; subnormal, zero, infinite and NaN groups."""
    mid = np.concatenate([GRID, (GRID[1:] + GRID[:-1]) / 2])
    v = np.concatenate([mid, mid * (1 + 2.0 ** -7), mid * (1 - 2.0 ** -8), [0.1, 5.0, 6.0, 5.5]])
    v = np.minimum(np.concatenate([v, -v]), 6)
    w = np.zeros((32, 128))
    for n in range(128):
        w[0, n] = 6.0 * 2.0 ** (n % 40 - 20)
        w[1:, n] = np.roll(v, 7 * n)[:31] * 2.0 ** (n % 40 - 20)
    w[:, 100] = 0
    w[:, 101] *= 2.0 ** -110
    w[3, 102] = -np.inf
    w[4, 103] = np.nan
    w[:, 104] = np.sign(w[:, 104]) * 3.3e38
    fin = np.isfinite(w)
    w = np.where(fin, to_bf16(np.where(fin, w, 0)), w)
    got, want = host(tsf.prepare_fp4_weight(up(w)).dequantize()), fp4_held(w)
    # 3.3e38 is 3.88 of 2^126, held as 4: 2^128, to bf16 an infinity
    want = np.where(np.abs(want) >= 2.0 ** 128, np.copysign(np.inf, want), want)
    bad = ~((got == want) | (np.isnan(got) & np.isnan(want)))
    assert not bad.any(), (np.argwhere(bad)[:4], got[bad][:4], want[bad][:4])


def stored8(x):
    """held, by rows of many blocks at once."""
    x = np.asarray(x)
    if not np.isfinite(x).all():
        return held(x)
    m, k = x.shape
    p = np.zeros((m, -(-k // 128) * 128))
    p[:, :k] = x
    p = p.reshape(m, -1, 128)
    a = np.abs(p).max(2, keepdims=True)
    f, e = np.frexp(np.where(a > 0, a, 1.0))
    b = np.where(a > 0, np.clip(9 - e - (f > 0.875), -126, 126), 0)       # 448 = 0.875 2^9
    y = p * 2.0 ** b
    gap = 2.0 ** (np.maximum(np.frexp(np.where(y == 0, 1.0, y))[1] - 1, -6) - 3)
    return (np.round(y / gap) * gap * 2.0 ** -b).reshape(m, -1)[:, :k]


def test_stored8_is_held():
    g = np.random.Generator(np.random.PCG64(1))
    x = to_bf16(g.standard_normal((9, 300)) * np.exp2(g.integers(-9, 9, size=(9, 300))))
    assert np.array_equal(stored8(x), held(x))


def check(x, w, y):
    a, b = stored8(x), fp4_held(w)
    want = a @ b
    got = host(y)
    assert got.shape == want.shape
    bad = ~(np.abs(got - want) <= BF16_HALF * np.abs(want) + MFMA * (np.abs(a) @ np.abs(b)) + 2.0 ** -133)
    assert not bad.any(), (bad.sum(), np.argwhere(bad)[:3], got[bad][:3], want[bad][:3])


@pytest.mark.parametrize("M,K,N", [(1, 128, 16), (1, 1, 1), (1, 7, 300), (2, 8, 5), (1, 1111, 777), (3, 2048, 130),
                                   (4, 5000, 33), (16, 2048, 64), (7, 4700, 257), (13, 700, 1500), (1, 640, 9000),
                                   (17, 130, 500), (31, 1100, 410), (33, 500, 420), (64, 512, 200), (65, 1000, 129),
                                   (130, 1300, 300), (300, 260, 520), (257, 2100, 64)])
def test_linear(M, K, N):
    g = np.random.Generator(np.random.PCG64(M * K + N))
    x = to_bf16(g.standard_normal((M, K)) * np.exp2(g.integers(-6, 6, size=(M, 1))))
    w = weight(g, K, N)
    q = tsf.prepare_fp4_weight(up(w))
    y = tsf.fp4_linear_fwd_cached(up(x), q)
    check(x, w, y)
    wide = torch.full((M, K + 3), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[:, 1:K + 1] = up(x)
    out = torch.empty((M, N), dtype=torch.bfloat16, device="cuda")
    assert tsf.fp4_linear_fwd_cached(wide[:, 1:K + 1], q, out) is out
    assert torch.equal(out, y)                                             # any pitch, the same bits


# (form, row tiles, column tiles, groups over K) and rows and columns that choose them
FORMS = {
    (0, 1, 1, 1): (3, 70), (0, 1, 2, 1): (1, 4120), (0, 1, 3, 1): (2, 8200),
    (1, 1, 1, 1): (16, 90), (1, 1, 2, 1): (16, 4120), (1, 1, 3, 1): (15, 8200), (1, 2, 1, 1): (21, 16), (1, 2, 2, 1): (32, 4120),
    (1, 2, 3, 1): (21, 8200), (1, 4, 1, 1): (36, 50), (1, 4, 2, 1): (64, 4120), (1, 4, 3, 1): (50, 8200),
    (2, 4, 1, 2): (65, 16), (2, 5, 1, 2): (65, 8200), (2, 6, 1, 2): (83, 8200), (2, 7, 1, 2): (101, 8200),
    (2, 4, 2, 2): (113, 8200), (2, 5, 2, 2): (65, 16600), (2, 6, 2, 2): (257, 9880), (2, 7, 2, 2): (197, 12520),
    (2, 8, 2, 2): (245, 12520), (2, 4, 3, 2): (83, 16600), (2, 5, 3, 2): (131, 16600), (2, 6, 3, 2): (161, 16600),
    (2, 7, 3, 2): (197, 16600), (2, 8, 3, 2): (245, 16600), (2, 4, 2, 1): (293, 12520), (2, 5, 2, 1): (227, 16600),
    (2, 6, 2, 1): (257, 19720), (2, 7, 2, 1): (323, 16600), (2, 8, 2, 1): (341, 19720), (2, 4, 3, 1): (257, 16600),
    (2, 5, 3, 1): (341, 16600), (2, 6, 3, 1): (401, 16600), (2, 7, 3, 1): (600, 14680), (2, 8, 3, 1): (500, 19720),
    (3, 4, 1, 2): (65, 1), (3, 4, 2, 1): (164, 16480), (3, 4, 2, 2): (119, 8193), (3, 4, 3, 1): (83, 32800), (3, 4, 3, 2): (83, 16480),
    (3, 5, 1, 2): (65, 8193), (3, 5, 2, 1): (200, 16480), (3, 5, 2, 2): (65, 16480), (3, 5, 3, 1): (137, 32800), (3, 5, 3, 2): (65, 32800),
    (3, 6, 1, 2): (83, 8193), (3, 6, 2, 1): (263, 19880), (3, 6, 2, 2): (83, 24640), (3, 7, 1, 2): (101, 8193), (3, 7, 2, 1): (200, 24640),
    (3, 7, 2, 2): (200, 12400), (3, 8, 2, 1): (245, 24640), (3, 8, 2, 2): (119, 24640)}


def is_exact(form):
    """Asked for as exact: the exact form of many rows, and that of few from 33 on."""
    return form[0] == 3 or form[:2] == (1, 4)


def blocks_of(form):
    """K: from one block of 128 to ten, ends within one; above 16 blocks a row, so that few rows are not fused."""
    if form[0] == 1:
        return 2000 + 37 * sum(form)
    return (90, 200, 385, 640, 777, 1200)[(form[1] + form[2] + form[3]) % 6]


@pytest.mark.parametrize("form", list(FORMS), ids=str)
def test_every_form(form):
    M, N = FORMS[form]
    K = blocks_of(form)
    g = np.random.Generator(np.random.PCG64(M + N))
    x = to_bf16(g.standard_normal((M, K)) * np.exp2(g.integers(-6, 6, size=(M, 1))))
    w = weight(g, K, N)
    y = tsf.fp4_linear_fwd_cached(up(x), tsf.prepare_fp4_weight(up(w)), exact=is_exact(form))
    check(x, w, y)
    if form[0] == 2:
        return
    # exact products: sqrt(K) roundings of 2^-24 of the sum move an output to the next bf16 value, 2^-8 away, in
    # sqrt(2400) 2^-16 = 7.5e-4 of the cases (the 8-bit instructions, 1.5e-5 off, in 4e-3)
    off = host(y) != to_bf16(stored8(x) @ fp4_held(w))
    assert off.sum() <= 1 + 1e-3 * off.size, off.mean()


def test_rows_are_alike():
    """exact: a row has the same bits beside any number of others of the same form."""
    g = np.random.Generator(np.random.PCG64(12))
    x, w = up(g.standard_normal((300, 640))), tsf.prepare_fp4_weight(up(weight(g, 640, 260)))
    y = tsf.fp4_linear_fwd_cached(x, w, exact=True)
    assert torch.equal(tsf.fp4_linear_fwd_cached(x[100:], w, exact=True), y[100:])


@pytest.mark.parametrize("exact", [False, True])
@pytest.mark.parametrize("M", [1, 20, 200])
def test_linear_nonfinite(M, exact):
    """A NaN of X stays in its row, one of W in its column; an infinity of X saturates its block."""
    g = np.random.Generator(np.random.PCG64(6))
    K, N = 700, 210
    x, w = to_bf16(g.standard_normal((M, K))), weight(g, K, N)
    x[M - 1, 5] = np.inf
    check(x, w, tsf.fp4_linear_fwd_cached(up(x), tsf.prepare_fp4_weight(up(w)), exact=exact))
    x[0, 699], w[300, 77] = np.nan, np.nan
    y = tsf.fp4_linear_fwd_cached(up(x), tsf.prepare_fp4_weight(up(w)), exact=exact)
    nan = torch.zeros((M, N), dtype=torch.bool, device="cuda")
    nan[0], nan[:, 77] = True, True
    assert torch.equal(torch.isnan(y), nan)


def test_empty():
    bf = dict(dtype=torch.bfloat16, device="cuda")
    w = tsf.prepare_fp4_weight(torch.ones((64, 48), **bf))
    assert tsf.fp4_linear_fwd_cached(torch.ones((0, 64), **bf), w).shape == (0, 48)
    w = tsf.prepare_fp4_weight(torch.ones((0, 48), **bf))
    for M in (3, 20, 70, 1000):
        y = torch.full((M, 48), 5.0, **bf)
        assert (tsf.fp4_linear_fwd_cached(torch.ones((M, 0), **bf), w, y) == 0).all()
    w = tsf.prepare_fp4_weight(torch.ones((64, 0), **bf))
    assert tsf.fp4_linear_fwd_cached(torch.ones((3, 64), **bf), w).shape == (3, 0)
    assert w.dequantize().shape == (64, 0)


def test_in_a_graph_and_module():
    g = np.random.Generator(np.random.PCG64(7))
    K, N = 900, 600
    lin = tsf.FP4InferenceLinear(up(weight(g, K, N)))
    x = up(g.standard_normal((2, 3, K)))
    lin(x)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = lin(x)
    for _ in range(3):
        new = up(g.standard_normal((2, 3, K)))
        want = lin(new)
        x.copy_(new)
        graph.replay()
        torch.cuda.synchronize()
        assert y.shape == (2, 3, N) and torch.equal(y, want)
    state = lin.state_dict()
    other = tsf.FP4InferenceLinear(torch.zeros((K, N), dtype=torch.bfloat16, device="cuda"))
    other.load_state_dict(state)
    assert torch.equal(other(x), want)
