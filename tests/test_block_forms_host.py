"""What the GPU tests of the block-scaled product reach, by the library's own
choice of tiles (no GPU): every tile, split and not, with every number of
k-blocks modulo its loop's unrolling. A change of the choice that leaves a form
untested fails here."""
import ctypes

import tensor_scaled_fp8_amd as tsf
from tensor_scaled_fp8_amd import _lib
from tests import test_gpu_block_forms, test_gpu_block_tiles

UNROLL = {(256, 256): 6, (256, 128): 6, (128, 128): 4, (128, 64): 4, (64, 64): 4}


def plan(M, N, R):
    v = [ctypes.c_int() for _ in range(3)]
    assert tsf.load().fp8_block_gemm_plan(M, N, R, *map(ctypes.byref, v)) == 0
    return tuple(x.value for x in v)


def forms(M, N, R):
    m, n, splits = plan(M, N, R)
    tiles, nk = -(-M // m) * -(-N // n), -(-R // 128)
    whole = tiles if splits == 1 else tiles // 256 * 256
    reached = {(m, n, nk % UNROLL[m, n])} if whole else set()
    return reached | ({(m, n, "split")} if whole < tiles else set())


def test_every_form_is_tested():
    want = {(m, n, r) for (m, n), u in UNROLL.items() for r in (*range(u), "split")}
    have = set().union(*(forms(*z) for z in test_gpu_block_tiles.SIZES + test_gpu_block_forms.SIZES))
    assert want <= have, sorted(want - have, key=str)
    # in all pairs of formats
    assert {plan(*z)[:2] for z in test_gpu_block_forms.SIZES} == set(UNROLL)


def test_whole_and_split_tiles_in_one_product():
    assert any(s > 1 and -(-M // m) * -(-N // n) > 256 for M, N, R in test_gpu_block_tiles.SIZES
               for m, n, s in [plan(M, N, R)])


def test_plan_query():
    f = tsf.load().fp8_block_gemm_plan
    none = (None, None, None)
    assert f(300, 300, 300, *none) == _lib.FP8_OK and f(0, 5, 0, *none) == _lib.FP8_OK
    for at in range(3):
        size = [4, 4, 4]
        size[at] = -1
        assert f(*size, *none) == _lib.FP8_ERR_INVALID
        size[at] = 1 << 23
        assert f(*size, *none) == _lib.FP8_ERR_UNSUPPORTED
    # its splits are what the workspace is for
    for z in test_gpu_block_tiles.SIZES:
        m, n, s = plan(*z)
        tiles = -(-z[0] // m) * -(-z[1] // n)
        want = tiles % 256 * s * m * n * 4 if s > 1 else 0
        assert tsf.load().fp8_block_gemm_workspace_bytes(*z) == want
