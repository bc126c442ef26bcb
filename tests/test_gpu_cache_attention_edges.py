"""Attention over the paged 8-bit cache where its numbers end: against the
definition in 64 bits at the values that the cache holds."""
import numpy as np
import pytest
import torch

import tensor_scaled_fp8_amd as tsf
from tests.test_gpu_cache import draw, host, ints, up
from tests.test_gpu_cache_attention import compare, filled

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("new,hq", [(1, 2), (5, 8), (40, 2)])
@pytest.mark.parametrize("scale,softcap", [(0.0, 0.0), (-0.0, 0.0), (0.0, 30.0), (0.0, 1000.0)])
def test_scale_of_zero(new, hq, scale, softcap):
    """0 times a query that is not finite is NaN, of its own head and row alone; of the others it is 0: the mean of values."""
    g = np.random.Generator(np.random.PCG64(new))
    cache, model, tables = filled(g, [50], 2, 64, 16)
    q = draw(g, (new, hq, 64), 1)
    q[0, 1, 5], q[new // 2, 0, 63] = np.nan, -np.inf
    out = compare(q, cache, model, tables, [50], [0, new], scale=scale, softcap=softcap)
    bad = torch.zeros((new, hq), dtype=torch.bool)
    bad[0, 1] = bad[new // 2, 0] = True
    assert torch.equal(torch.isnan(out).all(2).cpu(), bad) and torch.equal(torch.isnan(out).any(2).cpu(), bad)
    # where nothing is seen it makes no difference
    none = tsf.fp8_cache_attention(up(q), cache, ints(np.full_like(tables, -1)), ints([50]), ints([0, new]), scale=scale, lse=True)
    assert (none[0] == 0).all() and (none[1] == -np.inf).all()
