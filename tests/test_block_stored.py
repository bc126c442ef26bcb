"""Stored matrices whose data do not go with their sizes are refused before
anything is launched (no GPU): the kernels read codes and scales by the sizes."""
import pytest
import torch

import tensor_scaled_fp8_amd as tsf
from tensor_scaled_fp8_amd import block

ROWS, COLS = 5, 130
N = ROWS * 256 + 128 * 2


def _data(n=N, dtype=torch.uint8):
    return torch.zeros(n, dtype=dtype)


BAD = {"short": _data(N - 1), "long": _data(N + 1), "codes only": _data(ROWS * 256), "none": _data(0),
       "another type": _data(N, torch.int8), "as 16-bit words": _data(N // 2, torch.int16),
       "every other byte": _data(2 * N)[::2]}


def test_right_data():
    q = tsf.BlockTensor(_data(), ROWS, COLS, "e5m2")
    assert q.nbytes == N and q.fmt == 1 and q.codes.shape == (ROWS, 256) and q.scales.shape == (2, 128)
    assert tsf.BlockTensor(_data(0), 0, 7, 0).shape == (0, 7)


@pytest.mark.parametrize("bad", list(BAD) + ["2-D"])
def test_construction(bad):
    d = _data().view(2, -1) if bad == "2-D" else BAD[bad]
    with pytest.raises(ValueError, match="contiguous bytes"):
        tsf.BlockTensor(d, ROWS, COLS, 0)


def test_construction_sizes_and_format():
    for rows, cols in ((-1, 4), (4, -1), (-128, -128)):
        with pytest.raises(ValueError, match="negative"):
            tsf.BlockTensor(_data(), rows, cols, 0)
    with pytest.raises(ValueError, match="unknown FP8 format"):
        tsf.BlockTensor(_data(), ROWS, COLS, 7)


@pytest.mark.parametrize("bad", list(BAD))
def test_use(bad):
    """Data exchanged after construction, and data that the module's buffer holds, are checked where they are used."""
    q, ok = (tsf.BlockTensor.empty(ROWS, COLS, "e4m3", "cpu") for _ in range(2))
    q.data = BAD[bad]
    for a, b in ((q, ok), (ok, q)):
        with pytest.raises(ValueError, match="contiguous bytes|on the device"):
            tsf.fp8_block_gemm(a, b)
    with pytest.raises(ValueError, match="contiguous bytes"):
        tsf.fp8_block_gemm(q, ok)
    with pytest.raises(ValueError, match="contiguous bytes"):
        block._check_data(q.data, q.rows, q.cols, "q")
    compiled = block._binding()
    with pytest.raises(ValueError, match="contiguous bytes"):
        compiled.dequantize(q.data, ROWS, COLS, 0, None)
    with pytest.raises(ValueError, match="contiguous bytes"):
        compiled.serve(torch.zeros(2, COLS, dtype=torch.bfloat16), q.data, ROWS, None)
