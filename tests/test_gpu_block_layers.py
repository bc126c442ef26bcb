"""Store, restore and SwiGLU at sizes of whole layers, whose kernels take
several rows a thread, against the definition in 64 bits on bands of rows: the
first, ones inside and across the workgroups' rows, and the ragged last; odd
columns and odd pitches."""
import numpy as np
import pytest
import torch

import tensor_scaled_fp8_amd as tsf
from tests.block_util import BF16_HALF, MFMA, blocks, held, sigmoid

pytestmark = pytest.mark.gpu

ROWS, COLS = 4003, 4201                  # 32 x 33 tiles of 128 x 128
BANDS = ((0, 3), (126, 131), (2047, 2052), (ROWS - 4, ROWS))
TINY = 2.0 ** -133


def down(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def soft(g):
    """32-bit sigmoid: the exponential's argument rounded at |g| log2(e) 2^-24, a few operations of 2^-23 each."""
    return 2.0 ** -20 + np.abs(g) * 2.0 ** -22


def _wide(seed, extra, spread=0):
    """bf16 [ROWS, COLS] at an odd start in rows of an odd pitch; NaN around it."""
    g = torch.Generator("cuda").manual_seed(seed)
    x = torch.randn((ROWS, COLS), generator=g, device="cuda")
    if spread:
        x *= torch.exp2(torch.randint(-spread, spread + 1, (ROWS, 33), generator=g, device="cuda").float()
                        ).repeat_interleave(128, 1)[:, :COLS]
        x[torch.rand((ROWS, COLS), generator=g, device="cuda") < 0.05] = 0
    wide = torch.full((ROWS, COLS + extra), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[:, 1:COLS + 1] = x.to(torch.bfloat16)
    return wide[:, 1:COLS + 1]


@pytest.mark.parametrize("form", ["rows", "both"])
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_store_and_restore(fmt, form):
    x = _wide(1, 6, 20)
    x[2048, 130], x[2049, 131], x[ROWS - 1, COLS - 1] = float("inf"), float("nan"), float("-inf")
    q, qt = tsf.fp8_block_quantize(x, fmt, transposed=form == "both")
    out = torch.full((ROWS, COLS + 7), 7.0, dtype=torch.bfloat16, device="cuda")
    tsf.fp8_block_dequantize(q, out[:, 3:COLS + 3])
    biases = q.biases()
    for a, b in BANDS:
        m = down(x[a:b])
        codes, want = blocks(m, fmt)
        assert np.array_equal(biases[a:b].cpu().numpy(), want)
        got, want = q.codes[a:b].cpu().numpy(), codes
        nan = np.pad(np.isnan(m), ((0, 0), (0, codes.shape[1] - COLS)))      # a NaN's code may be any of the format's
        assert np.array_equal(got[~nan], want[~nan])
        assert np.array_equal(down(out[a:b, 3:COLS + 3]), held(m, fmt), equal_nan=True)
    assert (out[:, :3] == 7.0).all() and (out[:, COLS + 3:] == 7.0).all()
    if form == "both":
        biases = qt.biases()
        for a, b in ((0, 2), (129, 131), (COLS - 2, COLS)):
            codes, want = blocks(down(x[:, a:b]).T, fmt)
            nan = np.pad(np.isnan(down(x[:, a:b]).T), ((0, 0), (0, codes.shape[1] - ROWS)))
            assert np.array_equal(biases[a:b].cpu().numpy(), want)
            assert np.array_equal(qt.codes[a:b].cpu().numpy()[~nan], codes[~nan])


def test_swiglu():
    G, U, dh = _wide(2, 6).mul_(3), _wide(3, 2), _wide(4, 8).mul_(1e-3)
    G[2048, 5], G[ROWS - 1, 7] = -95.0, -120.0          # far gates among ordinary ones
    U[2048, 5], U[ROWS - 1, 7] = 1e30, 1e30
    gate, up = G.detach().requires_grad_(), U.detach().requires_grad_()
    h = tsf.swiglu(gate, up)
    dG, dU = torch.autograd.grad(h, (gate, up), dh)
    with torch.no_grad():
        assert torch.equal(tsf.swiglu(gate, up), h)
    for r0, r1 in BANDS:
        a, b, d = down(G[r0:r1]), down(U[r0:r1]), down(dh[r0:r1])
        want = a * sigmoid(a) * b
        assert (np.abs(down(h[r0:r1]) - want) <= (BF16_HALF + soft(a)) * np.abs(want) + TINY).all()
        p, q = held(a), held(b)
        s = sigmoid(p)
        want = d * p * s
        assert (np.abs(down(dU[r0:r1]) - want) <= (BF16_HALF + soft(p)) * np.abs(want) + TINY).all()
        want = d * q * s * (1 + p * (1 - s))
        tol = BF16_HALF * np.abs(want) + soft(p) * np.abs(d * q * s) * (1 + np.abs(p) * (1 - s)) + TINY
        assert (np.abs(down(dG[r0:r1]) - want) <= tol).all()


def test_swiglu_one_gradient():
    G, U, dh = _wide(5, 6), _wide(6, 2), _wide(7, 8)
    gate, up = G.detach().requires_grad_(), U.detach().requires_grad_()
    dG, dU = torch.autograd.grad(tsf.swiglu(gate, up), (gate, up), dh)
    assert torch.equal(torch.autograd.grad(tsf.swiglu(gate, U), gate, dh)[0], dG)
    assert torch.equal(torch.autograd.grad(tsf.swiglu(G, up), up, dh)[0], dU)


def test_mlp():
    """Whole numbers make the first product and dh exact (test_gpu_block.py);
    Y and dX on bands of rows, the weights' gradients on bands of columns."""
    M, K, F, near = 2050, 40, 8200, 2.0 ** -17
    r = np.random.Generator(np.random.PCG64(8))
    x = r.integers(-1, 2, size=(M, K)).astype(np.float64)
    wgu = r.integers(-1, 2, size=(K, 2 * F)) / 4.0
    wd = r.integers(-1, 2, size=(F, K)).astype(np.float64)
    dy = r.integers(-1, 2, size=(M, K)).astype(np.float64)

    def up(v):
        return torch.from_numpy(np.ascontiguousarray(v, dtype=np.float32)).cuda().to(torch.bfloat16)
    T = [up(v).requires_grad_() for v in (x, wgu, wd)]
    Y = tsf.block_mlp(*T)
    dX, dWgu, dWd = torch.autograd.grad(Y, T, up(dy))

    def check(got, pairs):
        want = sum(p @ w for p, _, w in pairs)
        tol = sum(MFMA * np.abs(p) @ np.abs(w) + u @ np.abs(w) for p, u, w in pairs)
        assert (np.abs(got - want) <= BF16_HALF * np.abs(want) + tol + TINY).all()

    def gradients(p, q, d):
        s = sigmoid(p)
        return d * q * s * (1 + p * (1 - s)), d * p * s
    for r0, r1 in ((0, 3), (1023, 1026), (M - 3, M)):
        gu, d = x[r0:r1] @ wgu, dy[r0:r1] @ wd.T
        a, b = gu[:, :F], gu[:, F:]
        check(down(Y[r0:r1]), [(*held(a * sigmoid(a) * b, slack=near), wd)])
        da, db = gradients(held(a), held(b), d)
        check(down(dX[r0:r1]), [(*held(da, "e5m2", near), wgu[:, :F].T), (*held(db, "e5m2", near), wgu[:, F:].T)])
    for block, pick in ((slice(0, 128), [0, 77, 127]), (slice(8192, F), [0, 7])):
        d = (dy @ wd[block].T)[:, pick]
        p, q = held(x @ wgu[:, :F][:, block])[:, pick], held(x @ wgu[:, F:][:, block])[:, pick]
        at = np.arange(F)[block][pick]
        da, db = gradients(p, q, d)
        for n, c in ((at, da), (F + at, db)):
            check(down(dWgu[:, torch.from_numpy(n)]).T, [(*held(c.T, "e5m2", near), x)])
        check(down(dWd[torch.from_numpy(at)]), [(*held((p * sigmoid(p) * q).T, slack=near), dy)])
