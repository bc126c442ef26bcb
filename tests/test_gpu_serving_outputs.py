"""Outputs that a caller gives to the serving operators count as changed in place."""
import numpy as np
import pytest
import torch

import tensor_scaled_fp8_amd as tsf
from tests.test_gpu_cache import ints, up

pytestmark = pytest.mark.gpu


def writes():
    """Each output by name: a tensor and the call that writes it."""
    g = np.random.Generator(np.random.PCG64(1))
    cache = tsf.BlockKVCache(2, 16, 2, 64, device="cuda")
    a = (ints([[0], [1]]), ints([3, 4]))
    k, v, q = (up(g.standard_normal((2, n, 64))) for n in (2, 2, 4))
    w, x = tsf.prepare_fp4_weight(up(g.standard_normal((64, 32)))), up(g.standard_normal((3, 64)))
    tsf.fp8_cache_append(cache, k, v, *a)

    def new(*shape):
        return up(g.standard_normal(shape))
    here, there, out, rk, rv, y = new(2, 4, 64), new(2, 4, 64), new(2, 4, 64), new(2, 2, 64), new(2, 2, 64), new(3, 32)
    return {"q rotated in place": (here, lambda: tsf.fp8_cache_append(cache, k, v, *a, q=here, q_out=here)),
            "q_out": (there, lambda: tsf.fp8_cache_append(cache, k, v, *a, q=q, q_out=there)),
            "out": (out, lambda: tsf.fp8_cache_attention(q, cache, *a, out=out)),
            "k": (rk, lambda: tsf.fp8_cache_read(cache, *a, k=rk)), "v": (rv, lambda: tsf.fp8_cache_read(cache, *a, v=rv)),
            "Y": (y, lambda: tsf.fp4_linear_fwd_cached(x, w, y)),
            "cache": (cache.data, lambda: tsf.fp8_cache_append(cache, k, v, *a))}


@pytest.mark.parametrize("name", ["q rotated in place", "q_out", "out", "k", "v", "Y", "cache"])
def test_a_backward_that_saved_them_is_refused(name):
    t, call = writes()[name]
    if t.dtype != torch.uint8:
        product = t * torch.ones((), device="cuda", requires_grad=True)         # saves t
        call()
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            product.sum().backward()
    before = t._version
    call()
    assert t._version > before


def test_inference_mode():
    """Tensors without a version are written as before, in and out of the mode."""
    with torch.inference_mode():
        made = writes()
        for _, call in made.values():
            call()
    for _, call in made.values():
        call()
    torch.cuda.synchronize()
