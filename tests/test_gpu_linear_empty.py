"""Linear on an empty batch under the gradient of a sum: the gradient (and here
the input) are expanded, with strides 0, and contiguous() leaves an empty tensor
as it is."""
import pytest
import torch

from fp8_scaled_quantization_scale_amd import linear
from gpu_util import need_gpu

pytestmark = pytest.mark.gpu

RECIPES = [linear.DelayedScaling, linear.Float8CurrentScaling, linear.Float8BlockScaling, linear.MXFP8BlockScaling,
           linear.Float8ChannelScaling]


@pytest.mark.parametrize("recipe", RECIPES)
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_gradients_of_nothing(recipe, dt):
    need_gpu()
    layer = linear.Linear(256, 128, recipe=recipe(), device="cuda")
    x = torch.zeros((), dtype=dt, device="cuda").expand(0, 256).detach().requires_grad_()
    y = layer(x)
    y.sum().backward()
    assert y.shape == (0, 128) and y.dtype == dt and x.grad.shape == (0, 256)
    assert layer.weight.grad.shape == (128, 256) and not layer.weight.grad.any()
