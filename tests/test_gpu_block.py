"""Block-scaled FP8 on the device against the definition in 64 bits
(tests/block_util.py): stored bytes exactly, products within their FP32
sums and one bf16 rounding, gradients against the formulas and against
differences."""
import numpy as np
import pytest
import torch

import tensor_scaled_fp8_amd as tsf
from tests.block_util import BF16_HALF, MFMA, blocks, held, sigmoid, to_bf16

pytestmark = pytest.mark.gpu

TINY = 2.0 ** -133          # bf16's smallest subnormal


def gen(seed):
    return np.random.Generator(np.random.PCG64(seed))


def up(x):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).cuda().to(torch.bfloat16)


def down(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def close(got, want, tol):
    got, want = down(got), np.asarray(want)
    assert got.shape == want.shape
    bad = ~(np.abs(got - want) <= tol)
    if bad.any():
        i = tuple(np.argwhere(bad)[0])
        raise AssertionError(f"{bad.sum()} of {bad.size} off; first at {i}: {got[i]} for {want[i]}")


def product_tol(a, b, want, more=0.0):
    return BF16_HALF * np.abs(want) + MFMA * (np.abs(a) @ np.abs(b).T) + more + TINY


def spread(g, shape):
    """bf16 values over many binades, with zeros and a zero block's worth of them."""
    x = g.standard_normal(shape) * np.exp2(g.integers(-20, 20, size=shape))
    x[g.random(shape) < 0.1] = 0
    return to_bf16(x)


# ---- store and restore -----------------------------------------------------------------

@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("rows,cols,pitch", [(1, 1, 1), (1, 128, 128), (3, 127, 131), (17, 129, 129), (128, 128, 136),
                                             (130, 300, 301), (257, 520, 520)])
def test_store_bytes(rows, cols, pitch, fmt):
    x = spread(gen(rows * cols), (rows, cols))
    if cols > 128:
        x[0, :128] = 0
    wide = torch.full((rows, pitch), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[:, :cols] = up(x)
    view = wide[:, :cols]
    for q, qt in (tsf.fp8_block_quantize(view, fmt, transposed=True),
                  (tsf.fp8_block_quantize(view, fmt)[0], tsf.fp8_block_quantize(view, fmt, False, True)[1])):
        for s, m in ((q, x), (qt, x.T)):
            codes, biases = blocks(m, fmt)
            assert np.array_equal(s.biases().cpu().numpy(), biases)
            # -0 and +0 are both zero: compare the values' bytes
            assert np.array_equal(s.codes.cpu().numpy(), codes)
        out = torch.full((rows, pitch), 7.0, dtype=torch.bfloat16, device="cuda")
        tsf.fp8_block_dequantize(q, out[:, :cols])
        assert np.array_equal(down(out[:, :cols]), held(x, fmt))
        assert (out[:, cols:] == 7.0).all()
        assert np.array_equal(down(qt.dequantize()), held(x.T, fmt))


def test_store_extremes():
    """Subnormal and largest bf16 values, significands at the borders of the scale rule, ties of the codes."""
    one = np.array([2.0 ** -133, 2.0 ** -126, 1.9921875 * 2.0 ** 127, 1.75, 1.7578125, 1.0, 17.0, 19.0, 0.0])
    x = np.zeros((len(one), 256))
    for i, v in enumerate(one):
        x[i, :128] = v * np.linspace(0, 1, 128).round(2)
        x[i, 127] = v
        x[i, 128 + i] = -v
    x = down(up(x))          # as bf16 holds them
    for fmt in ("e4m3", "e5m2"):
        q = tsf.fp8_block_quantize(up(x), fmt)[0]
        codes, biases = blocks(x, fmt)
        assert np.array_equal(q.biases().cpu().numpy(), biases)
        assert np.array_equal(q.codes.cpu().numpy(), codes)


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_store_nonfinite(fmt):
    """A block with an infinity or a NaN: scale 1, the infinity saturates, the NaN stays, other blocks are untouched."""
    x = spread(gen(5), (6, 384))
    x[1, 130], x[2, 131], x[3, 132], x[3, 133] = np.inf, np.nan, -np.inf, np.nan
    q, qt = tsf.fp8_block_quantize(up(x), fmt, transposed=True)
    for s, m in ((q, x), (qt, x.T)):
        codes, biases = blocks(m, fmt)
        assert np.array_equal(s.biases().cpu().numpy(), biases)
        got, want = down(s.dequantize()), held(m, fmt)
        assert np.array_equal(np.isnan(got), np.isnan(want))
        assert np.array_equal(got[~np.isnan(want)], want[~np.isnan(want)])


def test_store_empty_and_repeated_row():
    for shape in ((0, 5), (5, 0), (0, 0)):
        q, qt = tsf.fp8_block_quantize(torch.empty(shape, dtype=torch.bfloat16, device="cuda"), transposed=True)
        assert q.dequantize().shape == shape and qt.dequantize().shape == shape[::-1]
    x = spread(gen(6), (1, 200))
    q, qt = tsf.fp8_block_quantize(up(x).expand(9, 200), transposed=True)
    assert np.array_equal(down(q.dequantize()), np.repeat(held(x), 9, 0))
    assert np.array_equal(down(qt.dequantize()), held(np.repeat(x, 9, 0).T))
    with pytest.raises(ValueError, match="contiguous rows"):
        tsf.fp8_block_quantize(up(x).expand(9, 200).t())
    with pytest.raises(ValueError, match="2-D"):
        tsf.fp8_block_quantize(up(x)[0])
    with pytest.raises(ValueError, match="torch.bfloat16"):
        tsf.fp8_block_quantize(up(x).float())


# ---- product ---------------------------------------------------------------------------

SIZES = [(1, 1, 1), (1, 17, 129), (3, 130, 128), (16, 16, 256), (17, 5, 700), (64, 300, 1), (100, 129, 383),
         (128, 128, 1024), (129, 257, 640), (200, 131, 2000), (300, 520, 1500), (513, 260, 384), (33, 1030, 4096)]


@pytest.mark.parametrize("fa,fb", [("e4m3", "e4m3"), ("e5m2", "e4m3"), ("e4m3", "e5m2"), ("e5m2", "e5m2")])
@pytest.mark.parametrize("M,N,R", SIZES)
def test_gemm(M, N, R, fa, fb):
    g = gen(M + 7 * N + R)
    # scales that differ from block to block and row to row
    A = to_bf16(g.standard_normal((M, R)) * np.exp2(g.integers(-6, 6, size=(M, 1))) *
                np.exp2(np.repeat(g.integers(-8, 8, size=(M, -(-R // 128))), 128, 1)[:, :R]))
    B = to_bf16(g.standard_normal((N, R)) * np.exp2(np.repeat(g.integers(-8, 8, size=(N, -(-R // 128))), 128, 1)[:, :R]))
    a, b = tsf.fp8_block_quantize(up(A), fa)[0], tsf.fp8_block_quantize(up(B), fb)[0]
    wide = torch.full((M, N + 3), 5.0, dtype=torch.bfloat16, device="cuda")
    out = tsf.fp8_block_gemm(a, b, wide[:, :N])
    ha, hb = held(A, fa), held(B, fb)
    want = ha @ hb.T
    close(out, want, product_tol(ha, hb, want))
    assert (wide[:, N:] == 5.0).all()
    assert torch.equal(tsf.fp8_block_gemm(a, b), out)          # the same bits every time


def test_gemm_far_scales():
    """Row scales at both ends of their range, whose products are ordinary numbers."""
    g = gen(9)
    A, B = to_bf16(g.standard_normal((40, 256))), to_bf16(g.standard_normal((50, 256)))
    s = np.exp2(np.where(np.arange(256) < 128, 100.0, -100.0))
    a, b = tsf.fp8_block_quantize(up(A * s))[0], tsf.fp8_block_quantize(up(B / s))[0]
    ha, hb = held(A * s), held(B / s)
    want = ha @ hb.T
    close(tsf.fp8_block_gemm(a, b), want, product_tol(ha, hb, want))


def test_gemm_nan_stays_in_its_row():
    g = gen(10)
    A, B = to_bf16(g.standard_normal((140, 300))), to_bf16(g.standard_normal((70, 300)))
    A[3, 7], B[5, 290] = np.nan, np.nan
    out = down(tsf.fp8_block_gemm(tsf.fp8_block_quantize(up(A))[0], tsf.fp8_block_quantize(up(B))[0]))
    nan = np.zeros((140, 70), bool)
    nan[3], nan[:, 5] = True, True
    assert np.array_equal(np.isnan(out), nan)


def test_gemm_empty():
    def q(r, c):
        return tsf.fp8_block_quantize(torch.zeros((r, c), dtype=torch.bfloat16, device="cuda"))[0]
    assert tsf.fp8_block_gemm(q(0, 64), q(5, 64)).shape == (0, 5)
    out = torch.full((3, 5), 2.0, dtype=torch.bfloat16, device="cuda")
    assert (tsf.fp8_block_gemm(q(3, 0), q(5, 0), out) == 0).all()


def test_far_offsets():
    """Codes past 4 GiB: the last rows of a large matrix stored, multiplied and restored as on their own."""
    rows, cols = 66100, 65600
    x = torch.zeros((rows, cols), dtype=torch.bfloat16, device="cuda")
    tail = torch.randn((300, cols), device="cuda", generator=torch.Generator("cuda").manual_seed(3)).to(torch.bfloat16)
    x[-300:] = tail
    q = tsf.fp8_block_quantize(x)[0]
    del x
    own = tsf.fp8_block_quantize(tail)[0]
    assert torch.equal(q.codes[-300:], own.codes)
    w = tsf.fp8_block_quantize(torch.randn((130, cols), device="cuda").to(torch.bfloat16))[0]
    got, want = tsf.fp8_block_gemm(q, w)[-300:].float(), tsf.fp8_block_gemm(own, w).float()
    # sums of 65600 standard normal products in another order: 1e-4 of a sum of |a b| below 65600
    assert (got - want).abs().max() <= 2 * BF16_HALF * want.abs().max() + 2 * MFMA * cols
    assert torch.equal(q.dequantize()[-300:], own.dequantize())


# ---- linear ----------------------------------------------------------------------------

@pytest.mark.parametrize("M,K,N", [(1, 1, 1), (1, 300, 40), (5, 128, 129), (130, 257, 66), (256, 384, 512),
                                   (333, 130, 270)])
def test_linear(M, K, N):
    g = gen(M * K + N)
    x, w, dy = (to_bf16(g.standard_normal(s) * c) for s, c in (((M, K), 1), ((K, N), 0.05), ((M, N), 1e-4)))
    X, W = up(x).requires_grad_(), up(w).requires_grad_()
    Y = tsf.block_linear(X, W)
    dX, dW = torch.autograd.grad(Y, (X, W), up(dy))
    for got, a, b in ((Y, held(x), held(w.T)), (dX, held(dy, "e5m2"), held(w)), (dW, held(x.T), held(dy.T, "e5m2"))):
        want = a @ b.T
        close(got, want, product_tol(a, b, want))
    # one gradient at a time: the same bits
    Y2 = tsf.block_linear(X, W.detach())
    assert torch.equal(Y2, Y) and torch.equal(torch.autograd.grad(Y2, X, up(dy))[0], dX)
    Y3 = tsf.block_linear(X.detach(), W)
    assert torch.equal(Y3, Y) and torch.equal(torch.autograd.grad(Y3, W, up(dy))[0], dW)
    with torch.no_grad():
        assert torch.equal(tsf.block_linear(X, W), Y)
    w8 = tsf.prepare_block_weight(W.detach())
    y8 = tsf.fp8_block_linear_fwd_cached(X.detach(), w8)
    close(y8, held(x) @ held(w.T).T, product_tol(held(x), held(w.T), held(x) @ held(w.T).T))
    assert torch.equal(tsf.BlockInferenceLinear(W.detach())(X.detach()[None])[0], y8)


def test_linear_strides_and_leading_dims():
    g = gen(21)
    x, w, dy = (to_bf16(g.standard_normal(s)) for s in ((6, 70), (70, 50), (6, 50)))
    base = tsf.block_linear(up(x), up(w))
    X = up(np.pad(x, ((0, 0), (3, 2))))[:, 3:73].reshape(2, 3, 70)     # odd start
    assert torch.equal(tsf.block_linear(X, up(w)).reshape(6, 50), base)
    assert torch.equal(tsf.block_linear(up(x.T).t(), up(w.T).t()), base)   # columns contiguous
    Xg = up(x).reshape(2, 3, 70).requires_grad_()
    Wg = up(w).requires_grad_()
    Y = tsf.block_linear(Xg, Wg)
    dX, dW = torch.autograd.grad(Y, (Xg, Wg), up(dy.T).t().reshape(2, 3, 50))
    X2, W2 = up(x).requires_grad_(), up(w).requires_grad_()
    eX, eW = torch.autograd.grad(tsf.block_linear(X2, W2), (X2, W2), up(dy))
    assert dX.shape == (2, 3, 70) and torch.equal(dX.reshape(6, 70), eX) and torch.equal(dW, eW)
    # a gradient of repeated rows (stride 0), as a sum's backward gives
    Y = tsf.block_linear(X2, W2)
    one = torch.ones((1, 1), dtype=torch.bfloat16, device="cuda").expand(6, 50)
    a = torch.autograd.grad(Y, (X2, W2), one, retain_graph=True)
    b = torch.autograd.grad(Y, (X2, W2), one.contiguous())
    assert all(torch.equal(p, q) for p, q in zip(a, b))


@pytest.mark.parametrize("M,K,N", [(0, 40, 30), (7, 0, 30), (7, 40, 0), (0, 0, 0)])
def test_linear_empty(M, K, N):
    X = torch.zeros((M, K), dtype=torch.bfloat16, device="cuda", requires_grad=True)
    W = torch.zeros((K, N), dtype=torch.bfloat16, device="cuda", requires_grad=True)
    Y = tsf.block_linear(X, W)
    assert Y.shape == (M, N) and (Y == 0).all()
    dX, dW = torch.autograd.grad(Y, (X, W), torch.ones_like(Y))
    assert dX.shape == (M, K) and (dX == 0).all() and dW.shape == (K, N) and (dW == 0).all()
    with torch.no_grad():
        assert tsf.fp8_block_linear_fwd_cached(X, tsf.prepare_block_weight(W)).shape == (M, N)


def test_linear_gradient_against_differences():
    """At small whole numbers everything is exact, so a difference of the loss is its gradient."""
    g = gen(31)
    M, K, N = 20, 150, 37
    x, w, dy = (g.integers(-2, 3, size=s).astype(np.float64) for s in ((M, K), (K, N), (M, N)))
    X, W = up(x).requires_grad_(), up(w).requires_grad_()
    dX, dW = torch.autograd.grad(tsf.block_linear(X, W), (X, W), up(dy))
    assert np.abs(down(dX)).max() <= 256 and np.abs(down(dW)).max() <= 256       # exact in bf16

    def loss(x, w):
        y = down(tsf.block_linear(up(x), up(w)))
        assert np.abs(y).max() <= 256
        return float((y * dy).sum())
    base = loss(x, w)
    for _ in range(12):
        i, k, n = g.integers(M), g.integers(K), g.integers(N)
        e = np.zeros_like(x)
        e[i, k] = 1
        assert loss(x + e, w) - base == down(dX)[i, k]
        e = np.zeros_like(w)
        e[k, n] = 1
        assert loss(x, w + e) - base == down(dW)[k, n]


# ---- SwiGLU ----------------------------------------------------------------------------

# sigmoid's 32-bit arithmetic: the exponential's argument is rounded at
# |g| log2(e) 2^-24, and a few operations of 2^-23 each
def soft(g):
    return 2.0 ** -20 + np.abs(g) * 2.0 ** -22


@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 200), (7, 128), (33, 131), (130, 1111), (1500, 1300)])
def test_swiglu(rows, cols):
    g = gen(rows + cols)
    a, b, dh = (to_bf16(g.standard_normal((rows, cols)) * c) for c in (3, 2, 1e-3))
    both = up(np.concatenate((a, b), 1))
    G, U = both[:, :cols].detach().requires_grad_(), both[:, cols:].detach().requires_grad_()
    h = tsf.swiglu(G, U)
    want = a * sigmoid(a) * b
    close(h, want, (BF16_HALF + soft(a)) * np.abs(want) + TINY)
    dG, dU = torch.autograd.grad(h, (G, U), up(dh))
    p, q = held(a), held(b)
    s = sigmoid(p)
    wu, inner = dh * p * s, 1 + p * (1 - s)
    close(dU, wu, (BF16_HALF + soft(p)) * np.abs(wu) + TINY)
    wg = dh * q * s * inner
    close(dG, wg, BF16_HALF * np.abs(wg) + soft(p) * np.abs(dh * q * s) * (1 + np.abs(p) * (1 - s)) + TINY)
    assert torch.equal(torch.autograd.grad(tsf.swiglu(G, U.detach()), G, up(dh))[0], dG)
    assert torch.equal(torch.autograd.grad(tsf.swiglu(G.detach(), U), U, up(dh))[0], dU)
    with torch.no_grad():
        assert torch.equal(tsf.swiglu(G, U), h)


def test_swiglu_far_gates_and_nonfinite():
    a = np.array([[-3e38, -1000, -100, -80, 80, 1000, 3e38, 0.0, -0.0, np.nan, np.inf, 1.0]])
    b = np.array([[1.0, 2, 3, 4, 5, 6, 0.5, 7, 8, 1, 1, np.inf]])
    a, b = down(up(a)), down(up(b))
    with np.errstate(invalid="ignore"):
        want = a * sigmoid(a) * b
    got = down(tsf.swiglu(up(a), up(b)))
    ok = np.isfinite(want)
    # sigmoids below 32 bits' range are 0
    assert (np.abs(got - want)[ok] <= ((BF16_HALF + soft(np.minimum(np.abs(a), 100))) * np.abs(want) +
                                       np.abs(a * b) * 2.0 ** -125)[ok]).all()
    assert np.array_equal(np.isnan(got), np.isnan(want)) and got[0, 10] == got[0, 11] == np.inf


def test_swiglu_gradient_against_differences():
    """At gates and ups that 8 bits hold exactly, against central differences of the function."""
    g = gen(41)
    a = held(to_bf16(g.standard_normal((5, 140)) * 2))
    b = held(to_bf16(g.standard_normal((5, 140))))
    dh = to_bf16(g.standard_normal((5, 140)))
    G, U = up(a).requires_grad_(), up(b).requires_grad_()
    dG, dU = torch.autograd.grad(tsf.swiglu(G, U), (G, U), up(dh))
    e = 1e-5

    def f(a, b):
        return a * sigmoid(a) * b
    wg = dh * (f(a + e, b) - f(a - e, b)) / (2 * e)
    wu = dh * (f(a, b + e) - f(a, b - e)) / (2 * e)
    # the differences' own error: e^2 / 6 of the third derivative (below 1 |b|), rounding 1e-16 / e
    own = np.abs(dh) * (1 + np.abs(a)) * (1 + np.abs(b)) * 1e-9
    close(dG, wg, BF16_HALF * np.abs(wg) + soft(a) * np.abs(dh * b) * (1 + np.abs(a)) + own)
    close(dU, wu, (BF16_HALF + soft(a)) * np.abs(wu) + own)


def test_swiglu_broadcast_and_empty():
    G = up(spread(gen(43), (1, 150))).requires_grad_()
    U = up(spread(gen(44), (9, 150))).requires_grad_()
    h = tsf.swiglu(G.expand(9, 150), U)
    dG, dU = torch.autograd.grad(h, (G, U), torch.ones_like(h))
    G9 = G.detach().repeat(9, 1).requires_grad_()
    h9 = tsf.swiglu(G9, U)
    eG, eU = torch.autograd.grad(h9, (G9, U), torch.ones_like(h9))
    assert torch.equal(h, h9) and torch.equal(dU, eU) and torch.equal(dG, eG.sum(0, keepdim=True))
    for shape in ((0, 5), (5, 0), (2, 0, 3)):
        G = torch.zeros(shape, dtype=torch.bfloat16, device="cuda", requires_grad=True)
        h = tsf.swiglu(G, G)
        assert h.shape == shape and torch.autograd.grad(h, G, h)[0].shape == shape


# ---- MLP -------------------------------------------------------------------------------

NEAR = 2.0 ** -17          # how far 32-bit h and gradients may be from 64 bits (soft() at the gates here), relative


@pytest.mark.parametrize("M,K,F", [(1, 5, 1), (3, 130, 128), (130, 64, 256), (65, 150, 200), (200, 96, 333)])
def test_mlp(M, K, F):
    """Small whole numbers make the first product and dh exact; where h or a
    gradient lies next to a rounding border of its 8 bits, either side is taken."""
    g = gen(M + K + F)
    x = g.integers(-1, 2, size=(M, K)).astype(np.float64)
    wgu = g.integers(-1, 2, size=(K, 2 * F)) / 4.0
    wd = g.integers(-1, 2, size=(F, K)).astype(np.float64)
    dy = g.integers(-1, 2, size=(M, K)).astype(np.float64)
    T = [up(t).requires_grad_() for t in (x, wgu, wd)]
    Y = tsf.block_mlp(*T)
    got = torch.autograd.grad(Y, T, up(dy))
    gu = x @ wgu
    assert np.array_equal(gu, to_bf16(gu))
    a, b = gu[:, :F], gu[:, F:]
    h, uh = held(a * sigmoid(a) * b, slack=NEAR)
    want = h @ wd
    close(Y, want, product_tol(h, wd.T, want, uh @ np.abs(wd)))
    dh = dy @ wd.T
    assert np.array_equal(dh, to_bf16(dh))
    p, q = held(a), held(b)
    s = sigmoid(p)
    da, db = dh * q * s * (1 + p * (1 - s)), dh * p * s
    # the halves' blocks are apart
    (ra, ua), (rb, ub) = held(da, "e5m2", NEAR), held(db, "e5m2", NEAR)
    parts = ((ra, ua, wgu[:, :F]), (rb, ub, wgu[:, F:]))
    want = sum(r @ w.T for r, _, w in parts)
    tol = sum(MFMA * np.abs(r) @ np.abs(w).T + u @ np.abs(w).T for r, u, w in parts)
    close(got[0], want, BF16_HALF * np.abs(want) + tol + TINY)
    c, uc = held(np.concatenate((da, db), 1).T, "e5m2", NEAR)
    want = x.T @ c.T
    close(got[1], want, product_tol(x.T, c, want, np.abs(x).T @ uc.T))
    ht, ut = held((p * s * q).T, slack=NEAR)
    want = ht @ dy
    close(got[2], want, product_tol(ht, dy.T, want, ut @ np.abs(dy)))
    # any subset of the gradients: the same bits
    for pick in ((0,), (1,), (2,), (0, 2)):
        t = [v if i in pick else v.detach() for i, v in enumerate(T)]
        y = tsf.block_mlp(*t)
        assert torch.equal(y, Y)
        for i, d in zip(pick, torch.autograd.grad(y, [T[i] for i in pick], up(dy))):
            assert torch.equal(d, got[i])
    with torch.no_grad():
        assert torch.equal(tsf.block_mlp(*T), Y)


@pytest.mark.parametrize("M,K,F", [(0, 8, 8), (4, 0, 8), (4, 8, 0)])
def test_mlp_empty(M, K, F):
    T = [torch.zeros(s, dtype=torch.bfloat16, device="cuda", requires_grad=True) for s in ((M, K), (K, 2 * F), (F, K))]
    Y = tsf.block_mlp(*T)
    assert Y.shape == (M, K) and (Y == 0).all()
    for t, d in zip(T, torch.autograd.grad(Y, T, torch.ones_like(Y))):
        assert d.shape == t.shape and (d == 0).all()


def test_modules_train():
    """The modules' parameters receive gradients; a second backward of the same graph is refused."""
    torch.manual_seed(0)
    mlp, lin = tsf.BlockMLP(96, 160, device="cuda"), tsf.BlockLinear(96, 50, device="cuda")
    x = torch.randn((2, 7, 96), device="cuda").to(torch.bfloat16)
    y = lin(x + mlp(x))
    y.float().square().mean().backward()
    for p in (mlp.gate_up, mlp.down, lin.weight):
        assert p.grad.shape == p.shape and torch.isfinite(p.grad).all() and p.grad.abs().max() > 0
    y = lin(x)
    y.sum().backward()
    with pytest.raises(RuntimeError):
        y.sum().backward()


def test_other_stream():
    g = gen(51)
    x, w = to_bf16(g.standard_normal((150, 260))), to_bf16(g.standard_normal((260, 140)))
    want = tsf.block_linear(up(x), up(w))
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        X, W = up(x).requires_grad_(), up(w).requires_grad_()
        Y = tsf.block_linear(X, W)
        d = torch.autograd.grad(Y, (X, W), Y.detach())
    st.synchronize()
    assert torch.equal(Y, want)
    X, W = up(x).requires_grad_(), up(w).requires_grad_()
    Y = tsf.block_linear(X, W)
    assert all(torch.equal(p, q) for p, q in zip(d, torch.autograd.grad(Y, (X, W), Y.detach())))


def test_graph_replays():
    """A captured forward and backward of the MLP, replayed on new inputs with eager work in between."""
    g = gen(61)
    M, K, F = 70, 130, 256

    def inputs():
        return [up(to_bf16(g.standard_normal(s) * 0.3)) for s in ((M, K), (K, 2 * F), (F, K), (M, K))]
    held_ = [t.clone() for t in inputs()]

    def step(x, wgu, wd, dy):
        t = [v.detach().requires_grad_() for v in (x, wgu, wd)]
        y = tsf.block_mlp(*t)
        return (y.detach(), *torch.autograd.grad(y, t, dy))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(*held_)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(*held_)
    for _ in range(4):
        new = inputs()
        want = step(*new)
        for a, b in zip(held_, new):
            a.copy_(b)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, want):
            assert torch.equal(a, b)
