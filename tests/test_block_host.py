"""Host-side checks of the block-scaled entry points (no GPU, no launch):
refusals of the C ABI and of the binding, workspace sizes, scale order."""
import ctypes

import pytest
import torch

import tensor_scaled_fp8_amd as tsf
from tensor_scaled_fp8_amd import _lib

INV, UNS, OK = _lib.FP8_ERR_INVALID, _lib.FP8_ERR_UNSUPPORTED, _lib.FP8_OK
P = 4096          # an aligned fake address, never dereferenced
BIG = 1 << 40


def vp(x):
    return ctypes.c_void_p(x)


def test_sizes():
    lib = tsf.load()
    assert lib.fp8_block_codes_bytes(3, 129) == 3 * 256
    assert lib.fp8_block_scales_bytes(3, 129) == 128 * 2
    assert lib.fp8_block_codes_bytes(0, 5) == 0 and lib.fp8_block_scales_bytes(-1, 5) == 0
    assert lib.fp8_swiglu_kept_bytes(-1, 4) == 0
    assert lib.fp8_swiglu_kept_bytes(2, 128) == 4 * 256
    assert lib.fp8_block_gemm_workspace_bytes(-1, 2, 3) == 0
    a, b, c = (ctypes.c_size_t() for _ in range(3))
    r = [ctypes.byref(v) for v in (a, b, c)]
    assert lib.fp8_block_linear_bytes(5, 130, 7, 3, *r) == OK
    # X transposed [130, 5] and W [130, 7]: 130 x 128 codes, 256 scale bytes each
    assert a.value == 2 * (130 * 128 + 256)
    assert lib.fp8_block_linear_bytes(5, 130, 7, 0, *r) == OK and a.value == 0
    assert lib.fp8_block_linear_bytes(5, -1, 7, 0, *r) == INV
    assert lib.fp8_block_linear_bytes(5, 1, 7, 4, *r) == INV
    assert lib.fp8_block_linear_bytes(5, 1, 7, 0, None, r[1], r[2]) == INV
    assert lib.fp8_block_linear_bytes(1 << 23, 1, 7, 0, *r) == UNS
    assert lib.fp8_block_linear_bytes(1 << 20, 1 << 20, 7, 0, *r) == UNS
    assert lib.fp8_block_mlp_bytes(5, 130, 7, 7, *r) == OK and a.value > 0
    assert lib.fp8_block_mlp_bytes(5, 130, 7, 8, *r) == INV
    assert lib.fp8_block_mlp_bytes(5, 130, 1 << 23, 7, *r) == UNS


def test_quantize_refusals():
    q = tsf.load().fp8_block_quantize
    ok = [vp(P), 4, 8, 8, 0, vp(P), vp(P), None, None, None]
    for at, bad, want in ((0, None, INV), (0, vp(P + 1), INV), (1, -1, INV), (2, -1, INV), (3, -1, INV), (4, 2, INV),
                          (5, None, INV), (6, None, INV), (5, vp(P + 8), INV), (6, vp(P + 4), INV), (7, vp(P), INV),
                          (1, 1 << 23, UNS), (2, 1 << 23, UNS)):
        args = list(ok)
        args[at] = bad
        assert q(*args) == want, (at, bad)
    assert q(vp(P), 4, 8, 8, 0, None, None, None, None, None) == INV
    d = tsf.load().fp8_block_dequantize
    ok = [vp(P), vp(P), 4, 8, 0, vp(P), 8, None]
    for at, bad, want in ((0, None, INV), (1, vp(P + 2), INV), (2, -4, INV), (4, 5, INV), (5, vp(P + 1), INV),
                          (5, None, INV), (6, 7, INV), (3, 1 << 23, INV)):
        args = list(ok)
        args[at] = bad
        assert d(*args) == want, (at, bad)
    assert d(vp(P), vp(P), 1 << 23, 8, 0, vp(P), 8, None) == UNS


def test_gemm_refusals():
    g = tsf.load().fp8_block_gemm
    ok = [vp(P), vp(P), 0, vp(P), vp(P), 1, 4, 5, 6, vp(P), 5, None, 0, None]
    for at, bad, want in ((0, None, INV), (1, vp(P + 8), INV), (2, 2, INV), (3, vp(P + 1), INV), (4, None, INV),
                          (5, -1, INV), (6, -1, INV), (8, -6, INV), (9, None, INV), (9, vp(P + 1), INV), (10, 4, INV),
                          (11, vp(P + 4), INV), (8, 1 << 23, UNS)):
        args = list(ok)
        args[at] = bad
        assert g(*args) == want, (at, bad)


def test_linear_mlp_swiglu_refusals():
    lib = tsf.load()
    f = lib.fp8_block_linear_fwd
    ok = [vp(P), 8, vp(P), 6, 4, 8, 6, 3, vp(P), BIG, vp(P), BIG, vp(P), None]
    for at, bad in ((0, None), (0, vp(P + 1)), (1, -1), (2, None), (3, -1), (4, -4), (7, 4), (8, None), (8, vp(P + 8)),
                    (9, 10), (10, None), (11, 10), (12, None), (12, vp(P + 1))):
        args = list(ok)
        args[at] = bad
        assert f(*args) == INV, (at, bad)
    b = lib.fp8_block_linear_bwd
    ok = [vp(P), 6, 4, 8, 6, 3, vp(P), BIG, vp(P), BIG, vp(P), vp(P), None]
    for at, bad in ((0, None), (1, -1), (3, -1), (5, 8), (6, None), (7, 1), (8, None), (9, 1), (10, None), (11, None)):
        args = list(ok)
        args[at] = bad
        assert b(*args) == INV, (at, bad)
    c = lib.fp8_block_linear_fwd_cached
    ok = [vp(P), 8, 4, 8, 6, vp(P), vp(P), vp(P), BIG, vp(P), None]
    for at, bad in ((0, None), (1, -1), (2, -1), (5, None), (6, vp(P + 4)), (7, None), (8, 1), (9, None)):
        args = list(ok)
        args[at] = bad
        assert c(*args) == INV, (at, bad)
    s = lib.fp8_swiglu_fwd
    ok = [vp(P), 8, vp(P), 8, 4, 8, vp(P), vp(P), BIG, None]
    for at, bad in ((0, None), (1, -1), (2, vp(P + 1)), (4, -1), (6, None), (7, vp(P + 2)), (8, 100)):
        args = list(ok)
        args[at] = bad
        assert s(*args) == INV, (at, bad)
    s = lib.fp8_swiglu_bwd
    ok = [vp(P), 8, 4, 8, vp(P), BIG, vp(P), vp(P), None]
    for at, bad in ((0, None), (2, -1), (4, None), (5, 100), (6, vp(P + 1))):
        args = list(ok)
        args[at] = bad
        assert s(*args) == INV, (at, bad)
    assert s(vp(P), 8, 4, 8, vp(P), BIG, None, None, None) == INV
    m = lib.fp8_block_mlp_fwd
    ok = [vp(P), 8, vp(P), 6, vp(P), 8, 4, 8, 3, 7, vp(P), BIG, vp(P), BIG, vp(P), None]
    for at, bad in ((0, None), (2, None), (4, vp(P + 1)), (5, -1), (8, -3), (9, 8), (10, None), (11, 5), (12, None),
                    (13, 5), (14, None)):
        args = list(ok)
        args[at] = bad
        assert m(*args) == INV, (at, bad)
    m = lib.fp8_block_mlp_bwd
    ok = [vp(P), 8, 4, 8, 3, 7, vp(P), BIG, vp(P), BIG, vp(P), vp(P), vp(P), None]
    for at, bad in ((0, None), (1, -1), (5, 16), (6, None), (7, 5), (8, None), (9, 5), (10, None), (11, None), (12, None)):
        args = list(ok)
        args[at] = bad
        assert m(*args) == INV, (at, bad)


def test_binding_refusals():
    x = torch.zeros(4, 8, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="device tensor"):
        tsf.fp8_block_quantize(x)
    with pytest.raises(ValueError, match="device tensor"):
        tsf.block_linear(x, torch.zeros(8, 3, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="shape mismatch"):
        tsf.block_linear(x, torch.zeros(7, 3, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="shape mismatch"):
        tsf.swiglu(x, x[:3])
    with pytest.raises(ValueError, match="shape mismatch"):
        tsf.block_mlp(x, torch.zeros(8, 6, dtype=torch.bfloat16), torch.zeros(4, 8, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="device tensor"):
        tsf.swiglu(x, x)
    with pytest.raises(ValueError, match="device tensor"):
        tsf.prepare_block_weight(x)
    a, b = tsf.BlockTensor.empty(4, 8, "e4m3", "cpu"), tsf.BlockTensor.empty(4, 9, "e4m3", "cpu")
    with pytest.raises(ValueError, match="reduction mismatch"):
        tsf.fp8_block_gemm(a, b)
    with pytest.raises(ValueError, match="unknown FP8 format"):
        tsf.BlockTensor.empty(4, 8, "e3m4", "cpu")


def test_scale_order():
    """biases() undoes the order of the scale bytes that the header states."""
    rows, cols = 300, 260
    q = tsf.BlockTensor.empty(rows, cols, "e4m3", "cpu")
    assert q.codes.shape == (300, 384) and q.scales.shape == (3, 384)
    want = torch.randint(-126, 127, (rows, 3), generator=torch.Generator().manual_seed(1), dtype=torch.int32)
    for r in range(rows):
        for kb in range(3):
            q.scales[kb, (r & ~127) + 8 * (r % 16) + (r % 128) // 16] = 127 - int(want[r, kb])
    assert torch.equal(q.biases(), want)
