"""Host-side checks of the serving linear for few rows (no GPU, no launch)."""
import ctypes

import pytest

import tensor_scaled_fp8_amd as tsf
from tensor_scaled_fp8_amd import _lib

INV, UNS = _lib.FP8_ERR_INVALID, _lib.FP8_ERR_UNSUPPORTED
P = ctypes.c_void_p(4096)          # an aligned fake address, never dereferenced


def test_few():
    few = tsf.load().fp8_block_linear_few
    assert few(1, 32768, 8) == 1 and few(1, 32769, 8) == 0
    assert few(16, 2048, 8) == 1 and few(16, 2049, 8) == 0 and few(17, 1, 8) == 0
    assert few(-1, 8, 8) == 0 and few(1, 8, 1 << 23) == 0 and few(0, 0, 0) == 1


def test_few_refusals():
    f = tsf.load().fp8_block_linear_fwd_few
    ok = [P, 8, 4, 8, 6, P, P, P, None]
    odd = ctypes.c_void_p(4097)
    for at, bad, want in ((0, None, INV), (0, odd, INV), (1, -1, INV), (2, -4, INV), (4, -1, INV), (5, None, INV),
                          (6, ctypes.c_void_p(4100), INV), (7, None, INV), (7, odd, INV), (2, 17, UNS),
                          (3, 1 << 20, UNS), (4, 1 << 23, UNS)):
        args = list(ok)
        args[at] = bad
        assert f(*args) == want, (at, bad)


def test_stored_on_the_host_is_refused():
    q = tsf.BlockTensor.empty(4, 8, "e4m3", "cpu")
    with pytest.raises(ValueError, match="on the device"):
        q.dequantize()
    with pytest.raises(ValueError, match="on the device"):
        tsf.fp8_block_gemm(q, q)
