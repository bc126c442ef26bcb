"""SwiGLU at gates far below 0, where sigmoid leaves 32 bits and its product
with a large up does not: forward, gradients and the MLP's stored forms
against the formulas in 64 bits."""
import numpy as np
import pytest
import torch

import tensor_scaled_fp8_amd as tsf
from tests.block_util import BF16_HALF, MFMA, held, sigmoid, to_bf16

pytestmark = pytest.mark.gpu

TINY = 2.0 ** -133          # bf16's smallest subnormal


def up(x):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).cuda().to(torch.bfloat16)


def down(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def soft(g):
    """32-bit sigmoid: the exponential's argument rounded at |g| log2(e) 2^-24, a few operations of 2^-23 each."""
    return 2.0 ** -20 + np.abs(g) * 2.0 ** -22


GATES = np.concatenate((np.linspace(-400, -70, 90), -np.linspace(86, 90, 33), [-1000.0, -3e38, -80.5, 0.0, 0.5]))


@pytest.mark.parametrize("rows", [1, 20])
@pytest.mark.parametrize("size", [1.0, 1e10, 1e30, 3e38])
def test_forward(rows, size):
    a = down(up(np.tile(GATES, (rows, 1))))
    b = down(up(np.where(np.arange(a.size).reshape(a.shape) % 3 == 0, -size, size)))
    want = a * sigmoid(a) * b
    assert np.isfinite(want).all() and (np.abs(want) > 2.0 ** -126).any()
    got = down(tsf.swiglu(up(a), up(b)))
    assert (np.abs(got - want) <= (BF16_HALF + soft(np.maximum(a, -400))) * np.abs(want) + TINY).all()


def test_infinite_gate_and_neighbours():
    """0 times infinity stays a NaN, and an ordinary gate's bits do not depend on a far one beside it."""
    a = np.array([[-np.inf, -90.0, np.nan, 2.0, -1.0, np.inf, -500.0, 80.0]])
    b = np.array([[1.0, 1e30, 1.0, 3.0, 5.0, 2.0, 4.0, 1.0]])
    got = down(tsf.swiglu(up(a), up(b)))
    assert np.array_equal(np.isnan(got), [[True, False, True] + [False] * 5]) and got[0, 5] == np.inf
    assert got[0, 6] == 0 and abs(got[0, 1]) > 1e-8
    alone = down(tsf.swiglu(up(a[:, 3:5]), up(b[:, 3:5])))
    assert np.array_equal(got[:, 3:5], alone)


@pytest.mark.parametrize("rows", [1, 20])
@pytest.mark.parametrize("size,grad", [(1.0, 1.0), (1e30, 1e-3), (1e30, 1e6), (1e10, 1e20)])
def test_gradients(rows, size, grad):
    a = held(down(up(np.tile(np.concatenate((-np.linspace(70, 240, 120), [0.0, 1.0, -3.0])), (rows, 1)))))
    b, dh = held(np.full_like(a, to_bf16(size))), np.full_like(a, to_bf16(grad))
    b[:, ::3] *= -1
    dh[:, ::2] *= -1
    G, U = up(a).requires_grad_(), up(b).requires_grad_()
    assert np.array_equal(down(G), a)
    dG, dU = torch.autograd.grad(tsf.swiglu(G, U), (G, U), up(dh))
    s = sigmoid(a)
    wu, wg = dh * a * s, dh * b * s * (1 + a * (1 - s))
    assert (np.abs(wg) > 2.0 ** -126).any()
    assert (np.abs(down(dU) - wu) <= (BF16_HALF + soft(a)) * np.abs(wu) + TINY).all()
    tol = BF16_HALF * np.abs(wg) + soft(a) * np.abs(dh * b * s) * (1 + np.abs(a)) + TINY
    assert (np.abs(down(dG) - wg) <= tol).all()


def test_mlp():
    """Gates of -88 .. -120 and ups of 2^100: h is an ordinary number, and so are all gradients."""
    F, near = 130, 2.0 ** -15                # soft(-120) is below 2^-15
    g = np.random.Generator(np.random.PCG64(3))
    x = np.eye(3, 2)                         # rows 0 and 1 pick a gate row each, row 2 is 0
    gate = -8.0 * g.integers(11, 16, size=(2, F))
    ups = np.ldexp(g.integers(4, 8, size=(2, F)) / 4.0, 100)
    wgu, wd = np.concatenate((gate, ups), 1), g.integers(-1, 2, size=(F, 2)).astype(np.float64)
    dy = g.integers(1, 3, size=(3, 2)).astype(np.float64)
    assert np.array_equal(held(wgu.T).T, wgu) and np.array_equal(held(gate), gate) and np.array_equal(held(ups), ups)
    T = [up(t).requires_grad_() for t in (x, wgu, wd)]
    Y = tsf.block_mlp(*T)
    got = [down(t) for t in (Y, *torch.autograd.grad(Y, T, up(dy)))]
    gu = x @ wgu
    a, b = gu[:, :F], gu[:, F:]
    s = sigmoid(a)
    h, uh = held(a * s * b, slack=near)
    dh = dy @ wd.T
    da, db = dh * b * s * (1 + a * (1 - s)), dh * a * s
    assert (np.abs(h[:2]) > 2.0 ** -80).any() and (np.abs(da[:2]) > 2.0 ** -80).any()

    def check(out, pairs):
        want = sum(p @ w for p, _, w in pairs)
        tol = sum(MFMA * np.abs(p) @ np.abs(w) + u @ np.abs(w) for p, u, w in pairs)
        assert (np.abs(out - want) <= BF16_HALF * np.abs(want) + tol + TINY).all()
    check(got[0], [(h, uh, wd)])
    check(got[1], [(*held(d, "e5m2", near), w.T) for d, w in ((da, wgu[:, :F]), (db, wgu[:, F:]))])
    c, uc = held(np.concatenate((da, db), 1).T, "e5m2", near)
    check(got[2].T, [(c, uc, x)])
    ht, ut = held((a * s * b).T, slack=near)
    check(got[3], [(ht, ut, dy)])
