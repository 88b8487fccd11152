"""Dispatch and combine refuse what they have no derivative for, before any GPU
work: a dual tensor of forward-mode differentiation, whose tangent the kernels
do not carry."""
import pytest
import torch
from torch.autograd import forward_ad

import fp8_scaled_quantization_scale_amd as fm
from fp8_scaled_quantization_scale_amd import moe


def _plan():
    i = torch.zeros(8, dtype=torch.int32)
    return tuple.__new__(moe.Plan, (4, 2, 7, 8, i, i, i, i))


@pytest.mark.parametrize("call,rows", [(moe.dispatch, 4), (moe.combine, 8)])
@pytest.mark.parametrize("dual", ["rows", "weights"])
@pytest.mark.parametrize("grad", [False, True])
def test_forward_mode_is_refused(call, rows, dual, grad):
    x, w = torch.zeros(rows, 64), torch.ones(4, 2)
    with forward_ad.dual_level(), torch.set_grad_enabled(grad):
        if dual == "rows":
            x = forward_ad.make_dual(x, torch.ones_like(x))
        else:
            w = forward_ad.make_dual(w, torch.ones_like(w))
        with pytest.raises(fm.Fp8Error, match="no forward-mode derivative"):
            call(x, _plan(), w)


@pytest.mark.parametrize("call,rows", [(moe.dispatch, 4), (moe.combine, 8)])
def test_torch_func_jvp_is_refused(call, rows):
    x = torch.zeros(rows, 64)
    with pytest.raises(fm.Fp8Error, match="no forward-mode derivative"):
        torch.func.jvp(lambda v: call(v, _plan()), (x,), (torch.ones_like(x),))


@pytest.mark.parametrize("call,rows", [(moe.dispatch, 4), (moe.combine, 8)])
def test_tensors_without_a_tangent_pass(call, rows):
    """Inside a dual level too: these reach the check for device tensors."""
    with forward_ad.dual_level(), pytest.raises(fm.Fp8Error, match="device tensor"):
        call(torch.zeros(rows, 64), _plan(), torch.ones(4, 2))
