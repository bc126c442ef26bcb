"""Forward-mode derivatives of the block-scaled operators are refused (no GPU,
no launch): a result without its tangent would pass for a constant."""
import pytest
import torch
from torch.autograd import forward_ad

import tensor_scaled_fp8_amd as tsf


def _calls(x, w, wd):
    return {"linear": lambda: tsf.block_linear(x, w), "swiglu": lambda: tsf.swiglu(x, x),
            "mlp": lambda: tsf.block_mlp(x, w, wd)}


@pytest.mark.parametrize("name,dual", [("linear", "x"), ("linear", "w"), ("swiglu", "x"), ("mlp", "x"), ("mlp", "w"),
                                       ("mlp", "wd")])
def test_dual_tensors_are_refused(name, dual):
    t = {"x": torch.ones(4, 8), "w": torch.ones(8, 6), "wd": torch.ones(3, 8)}
    t = {k: v.to(torch.bfloat16) for k, v in t.items()}
    with forward_ad.dual_level():
        d = dict(t)
        d[dual] = forward_ad.make_dual(t[dual], t[dual])
        with pytest.raises(NotImplementedError, match="forward-mode"):
            _calls(**d)[name]()
        # a call inside the level that holds no tangent goes on to the ordinary checks
        with pytest.raises(ValueError, match="device tensor"):
            _calls(**t)[name]()


def test_jvp_is_refused():
    x, w = torch.ones(4, 8, dtype=torch.bfloat16), torch.ones(8, 6, dtype=torch.bfloat16)
    with pytest.raises(NotImplementedError, match="forward-mode"):
        torch.func.jvp(lambda v: tsf.block_linear(v, w), (x,), (x,))
