"""What the serving operators hold beyond a bf16's precision: softmax weights
in the forms that wait for the cache's bytes, and the products in front of the
cache's 8-bit roundings."""
import numpy as np
import pytest
import torch

import tensor_scaled_fp8_amd as tsf
from tests.serve_util import Model, attend, fp4_held
from tests.test_gpu_cache import draw, host, ints, tables_of, up
from tests.test_gpu_cache_attention import filled
from tests.test_gpu_fp4 import stored8
from tests.test_serving_precision import fine_tolerance

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("how", [dict(), dict(softcap=20.0, window=70)], ids=["plain", "cap-window"])
@pytest.mark.parametrize("heads,hq,d,lens,new", [
    (2, 8, 64, [300, 77], [1, 1]), (1, 4, 128, [500, 130], [1, 1]), (2, 4, 256, [200], [1]),              # 16 rows
    (2, 8, 64, [300, 70], [8, 8]), (1, 6, 128, [333], [5]), (1, 3, 256, [350], [9]),                       # 32
    (2, 4, 64, [300], [40]), (1, 8, 128, [260], [30]), (1, 1, 256, [150], [40])])                          # the most
def test_weights_in_two_parts(heads, hq, d, lens, new, how):
    """Equal shares: outputs are off by their own rounding and 2^-17 of what the weights weigh. A weight in one bf16 is not
    (tests/test_serving_precision.py)."""
    g = np.random.Generator(np.random.PCG64(hq * d + lens[0]))
    cache, model, tables = filled(g, lens, heads, d, 32)
    starts = np.concatenate([[0], np.cumsum(new)])
    q = host(up(0.1 * draw(g, (int(starts[-1]), hq, d), 1)))    # small scores: of large ones the products' roundings count
    got = host(tsf.fp8_cache_attention(up(q), cache, ints(tables), ints(lens), ints(starts), **how))
    want, _, mass, size = attend(q, model, tables, lens, starts, **how)
    bad = ~(np.abs(got - want) <= fine_tolerance(want, mass, size, d, max(lens), how.get("softcap", 0.0)))
    assert not bad.any(), (int(bad.sum()), bad.size, np.argwhere(bad)[:4], got[bad][:4], want[bad][:4])


def held_after(qkv, hq, hk, d, layer, x, lens):
    """A layer's cache after a call of whole prompts, and as it is by the definition from the exact projection."""
    starts = np.concatenate([[0], np.cumsum(lens)])
    tables, pages = tables_of(np.random.Generator(np.random.PCG64(1)), lens, 16)
    cache, model = tsf.BlockKVCache(pages, 16, hk, d, device="cuda"), Model(pages, 16, hk, d)
    layer(up(x), cache, ints(tables), ints(lens), ints(starts))
    a = host(up(qkv)).reshape(len(x), -1, d)
    model.append(a[:, hq:hq + hk], a[:, hq + hk:], tables, lens, starts)
    got = tsf.fp8_cache_read(cache, ints(tables), ints(lens), ints(starts), len(x))
    return np.stack([host(t) for t in got]), np.stack(model.read(tables, lens, starts))


@pytest.mark.parametrize("bits,rows,most", [(4, 140, 1e-4), (4, 50, 1e-4), (4, 12, 1e-4), (8, 140, 4e-3), (8, 12, 4e-3)])
def test_a_layers_cache(bits, rows, most):
    """Keys and values go to 8 bits behind their projection: an error next to a border of the 8-bit format becomes a step.

    4 bits: exact products, sums of K = 1024 in 32 bits: 32 roundings of 2^-24 / sqrt(3) at most of a partial sum of about the
    result's size, 2e-7 of it. A value changes where it lies within that of one of the two bf16 borders beside a border of the
    8-bit format, 8 of which share an octave: 2 * 2 * 2e-7 / 0.09, 9e-6 of the values; ten times that is allowed. The FP8
    instructions' sums (1.5e-5 of eight neighbours' largest) change more: 2.3e-4 of 140 rows without the exact products, and
    of 8-bit weights, which have no exact form, 1 in 1000, as the class says: four times that is allowed."""
    g = np.random.Generator(np.random.PCG64(bits * 1000 + rows))
    K, hq, hk, d = 1024, 4, 4, 128
    x = host(up(g.standard_normal((rows, K))))
    wqkv, wo = (host(up(g.standard_normal(s) * s[0] ** -0.5)) for s in ((K, (hq + 2 * hk) * d), (hq * d, K)))
    layer = tsf.InferenceAttention(up(wqkv), up(wo), hq, hk, d, bits=bits)
    exact = stored8(x) @ (fp4_held(wqkv) if bits == 4 else stored8(wqkv.T).T)
    got, want = held_after(exact, hq, hk, d, layer, x, [rows - 5, 5])
    assert (got != want).mean() <= most, (got != want).mean()
    # what differs differs by a step of the block's scale: 2^-3 of it, below its normal range 2^-9 of 2^-6
    assert (np.abs(got - want) <= 2.0 ** -3 * np.maximum(np.abs(got), np.abs(want)) + 2.0 ** -15 * np.abs(want).max()).all()
