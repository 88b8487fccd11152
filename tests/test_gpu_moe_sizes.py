"""Dispatch, combine and its gradient of more tokens than one launch holds
(2^32 work-items).

The values are small whole numbers, so that every product and sum below is
exact in binary32 whatever its order, and the results are compared bit for bit."""
import pytest
import torch

from fp8_scaled_quantization_scale_amd import moe
from gpu_util import need_gpu

pytestmark = pytest.mark.gpu

B = torch.bfloat16


def _one_expert(tokens):
    """Every token to one expert: row t of the sorted buffer is token t."""
    return moe.sort(torch.zeros(tokens, 1, dtype=torch.int32, device="cuda"), 1)


def _numbers(n, most):
    """-most .. most, again and again"""
    return (torch.arange(n, dtype=torch.int32, device="cuda") % (2 * most + 1) - most).to(B)


def test_more_tokens_than_one_grid_of_waves_holds():
    """A wave per token: 2^32 work-items are 2^26 tokens."""
    need_gpu()
    tokens = (1 << 26) + 1003
    plan = _one_expert(tokens)
    x = _numbers(tokens, 125)[:, None] + torch.arange(8, device="cuda", dtype=B)
    y = moe.dispatch(x, plan)
    assert torch.equal(y[:tokens], x) and not y[tokens:].any()
    assert torch.equal(moe.combine(y, plan), x)
    dys, dw = moe.combine_backward(x, y, plan, None)
    assert torch.equal(dys[:tokens], x) and not dys[tokens:].any()
    assert torch.equal(dw, x.float().square().sum(1, keepdim=True))


def test_more_tokens_than_one_grid_of_workgroups_holds():
    """A workgroup of 512 per token (rows over 2048 columns): 2^23 tokens."""
    need_gpu()
    tokens, cols = (1 << 23) + 5, 2049
    plan = _one_expert(tokens)
    ys = torch.empty(plan.rows, cols, dtype=B, device="cuda")
    v = _numbers(plan.rows, 7)
    ys.copy_(v[:, None].expand(-1, cols))
    dys, dw = moe.combine_backward(ys[:tokens], ys, plan, None)
    assert torch.equal(dys[:tokens], ys[:tokens]) and not dys[tokens:].any()
    assert torch.equal(dw[:, 0], cols * v[:tokens].float().square())
