"""Empty batches whose tensors have other strides than a row-major one's: the
gradient of a sum is expanded, with strides 0, and contiguous() leaves an empty
tensor as it is."""
import pytest
import torch

from fp8_scaled_quantization_scale_amd import linear, moe, norm
from gpu_util import need_gpu

pytestmark = pytest.mark.gpu

RECIPES = [linear.Float8BlockScaling(), linear.MXFP8BlockScaling()]


def _zero(like):
    assert like.grad.shape == like.shape and not like.grad.any()


def _empty(cols, dtype=torch.bfloat16):
    return torch.zeros((), dtype=dtype, device="cuda").expand(0, cols).detach().requires_grad_()


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_layer_norm(dt):
    need_gpu()
    layer = norm.LayerNorm(64, device="cuda")
    x = _empty(64, dt)
    layer(x).sum().backward()
    _zero(x), _zero(layer.weight), _zero(layer.bias)


@pytest.mark.parametrize("recipe", RECIPES, ids=["block", "mx"])
@pytest.mark.parametrize("gather", [False, True])
def test_grouped_linear(recipe, gather):
    need_gpu()
    layer = moe.GroupedLinear(3, 256, 128, recipe, device="cuda")
    plan = moe.sort(torch.empty(0, 2, dtype=torch.int64, device="cuda"), 3)
    x = _empty(256)
    layer(x, plan, gather=gather).sum().backward()
    _zero(x), _zero(layer.weight)


@pytest.mark.parametrize("call", [moe.dispatch, moe.combine])
def test_dispatch_and_combine(call):
    need_gpu()
    plan = moe.sort(torch.empty(0, 2, dtype=torch.int32, device="cuda"), 4)
    x = torch.empty(0, 96, device="cuda", requires_grad=True)
    w = torch.empty(0, 2, device="cuda", requires_grad=True)
    call(x, plan, w).sum().backward()
    _zero(x), _zero(w)


def test_block():
    """Layer norm, two grouped layers and the way back, under a gradient of a sum
    (strides 0)."""
    need_gpu()
    ln = norm.LayerNorm(256, device="cuda")
    up, down = (moe.GroupedLinear(4, *s, RECIPES[0], device="cuda") for s in ((256, 384), (384, 256)))
    x = torch.empty(0, 256, dtype=torch.bfloat16, device="cuda", requires_grad=True)
    w = torch.empty(0, 2, device="cuda", requires_grad=True)
    plan = moe.sort(torch.empty(0, 2, dtype=torch.int32, device="cuda"), 4)
    y = moe.combine(down(torch.relu(up(ln(x), plan, gather=True)), plan), plan, w)
    y.sum().backward()
    assert y.shape == x.grad.shape == (0, 256) and w.grad.shape == (0, 2)
    for p in (ln.weight, ln.bias, up.weight, down.weight):
        assert p.grad.shape == p.shape and not p.grad.any()
