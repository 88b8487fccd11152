"""The experts' layer on a batch without tokens, as a rank of expert
parallelism may have one: forward, and a backward pass whose weight gradient is
zero."""
import pytest
import torch

import fp8_scaled_quantization_scale_amd as fm
from fp8_scaled_quantization_scale_amd import linear, moe
from gpu_util import need_gpu

pytestmark = pytest.mark.gpu

RECIPES = [linear.Float8BlockScaling(), linear.MXFP8BlockScaling()]


@pytest.mark.parametrize("recipe", RECIPES, ids=["block", "mx"])
@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_layer(recipe, gather, dt):
    need_gpu()
    layer = moe.GroupedLinear(3, 256, 128, recipe, device="cuda")
    plan = moe.sort(torch.empty(0, 2, dtype=torch.int64, device="cuda"), 3)
    assert plan.rows == 0 and not plan.offsets.any() and not plan.counts.any()
    x = torch.empty(0, 256, dtype=dt, device="cuda", requires_grad=True)
    y = layer(x, plan, gather=gather)
    assert y.shape == (0, 128) and y.dtype == dt
    y.backward(torch.empty_like(y))
    assert x.grad.shape == (0, 256) and x.grad.dtype == dt
    assert layer.weight.grad.shape == layer.weight.shape and not layer.weight.grad.any()


@pytest.mark.parametrize("orient", [1, 2, 3])
def test_codes(orient):
    """The sorted codes of nothing have the sorted buffer's width."""
    need_gpu()
    plan = moe.sort(torch.empty(0, 1, dtype=torch.int64, device="cuda"), 2)
    q = moe.quantize(torch.empty(0, 64, dtype=torch.bfloat16, device="cuda"), plan, fm.BLOCK_1x128, fm.E4M3, orient)
    if orient & fm.ROW:
        assert q.q_row.shape == (0, 64) and q.s_row.shape == (0, 1)
    if orient & fm.COL:
        assert q.q_col.shape == (64, 0) and q.s_col.shape == (64, 0)
