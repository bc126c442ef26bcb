"""Autograd of the block-scaled operators beyond one backward: what their
compiled nodes cannot differentiate is refused, never taken for a constant."""
import pytest
import torch

import tensor_scaled_fp8_amd as tsf

pytestmark = pytest.mark.gpu


def _leaf(g, *shape):
    return torch.randn(shape, generator=g, device="cuda").to(torch.bfloat16).requires_grad_()


def _operators():
    g = torch.Generator("cuda").manual_seed(1)
    x, w, wd = _leaf(g, 5, 130), _leaf(g, 130, 140), _leaf(g, 70, 130)
    u = _leaf(g, 5, 130)
    return {"linear": (tsf.block_linear, (x, w)), "swiglu": (tsf.swiglu, (x, u)), "mlp": (tsf.block_mlp, (x, w, wd))}


@pytest.mark.parametrize("name", ["linear", "swiglu", "mlp"])
@pytest.mark.parametrize("seed", ["sum", "constant", "wanted"])
def test_gradient_of_a_gradient_is_refused(name, seed):
    """A penalty on dX depends on the other operands through dX: its share of
    their gradients must not go missing in silence, whatever the gradient
    that came in (a sum's expanded constant, a plain tensor, a leaf)."""
    f, leaves = _operators()[name]
    y = f(*leaves)
    if seed == "sum":
        d = torch.autograd.grad(y.sum(), leaves, create_graph=True)
    else:
        one = torch.ones_like(y).requires_grad_(seed == "wanted")
        d = torch.autograd.grad(y, leaves, one, create_graph=True)
    once = torch.autograd.grad(f(*leaves), leaves, torch.ones_like(y))
    for a, b in zip(d, once):
        assert torch.equal(a, b)                       # the values themselves can be read
    for i in range(len(leaves)):
        with pytest.raises(RuntimeError, match="once_differentiable"):
            (y.float().sum() + d[i].float().square().sum()).backward(retain_graph=True)


def test_create_graph_that_is_not_used():
    """backward(create_graph=True) of a model in which these gradients are only read."""
    f, leaves = _operators()["mlp"]
    f(*leaves).sum().backward(create_graph=True)
    want = torch.autograd.grad(f(*leaves), leaves, torch.ones_like(leaves[0]))
    for t, d in zip(leaves, want):
        assert torch.equal(t.grad, d)
        t.grad = None
