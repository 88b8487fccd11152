"""The RMS norm's and the router's C entry points refuse bad arguments before any
GPU work (only invalid and empty calls are made), and the bindings refuse host
tensors."""
import pytest
import torch

import fp8_scaled_quantization_scale_amd as fm
from fp8_scaled_quantization_scale_amd import linear, moe, norm

P = 0x10000  # an aligned stand-in pointer, never dereferenced
BIG = 1 << 62


def _fwd(**kw):
    a = dict(x=P, x_dtype=fm.IN_BF16, rows=8, cols=64, ld_x=64, residual=P, ld_residual=64, weight=P, w_dtype=fm.IN_FP32, eps=1e-6,
             total=P, ld_total=64, y=P, ld_y=64, rstd=P, stream=0)
    a.update(kw)
    return fm.fp8_rms_norm_forward(**a)


@pytest.mark.parametrize("kw,code", [
    (dict(x_dtype=2), fm.ERR_ENUM), (dict(w_dtype=-1), fm.ERR_ENUM), (dict(rows=-1), fm.ERR_SHAPE), (dict(cols=0), fm.ERR_SHAPE),
    (dict(cols=(1 << 28) + 1), fm.ERR_UNSUPPORTED), (dict(eps=-1e-9), fm.ERR_SHAPE), (dict(eps=float("nan")), fm.ERR_SHAPE),
    (dict(x=None), fm.ERR_NULL), (dict(y=None), fm.ERR_NULL), (dict(total=None), fm.ERR_NULL), (dict(rstd=None), fm.ERR_NULL),
    (dict(ld_x=63), fm.ERR_SHAPE), (dict(ld_y=63), fm.ERR_SHAPE), (dict(ld_residual=63), fm.ERR_SHAPE), (dict(ld_total=63), fm.ERR_SHAPE),
    (dict(ld_x=BIG), fm.ERR_SHAPE), (dict(x=P + 1), fm.ERR_ALIGN), (dict(y=P + 1), fm.ERR_ALIGN), (dict(residual=P + 1), fm.ERR_ALIGN),
    (dict(total=P + 1), fm.ERR_ALIGN), (dict(rstd=P + 2), fm.ERR_ALIGN), (dict(weight=P + 2), fm.ERR_ALIGN),
    (dict(x=P + 2, x_dtype=fm.IN_FP32), fm.ERR_ALIGN), (dict(rows=0, x=None, y=None, total=None, rstd=None), fm.OK),
])
def test_rms_forward(kw, code):
    assert _fwd(**kw) == code


def _quant(**kw):
    a = dict(x=P, x_dtype=fm.IN_BF16, rows=8, cols=64, ld_x=64, residual=P, ld_residual=64, weight=P, w_dtype=fm.IN_FP32, eps=1e-6,
             total=P, ld_total=64, rstd=P, recipe=fm.BLOCK_1x128, fmt=fm.E4M3, orient=fm.ROW_AND_COL, margin=0, q_row=P, ld_q_row=64,
             s_row=P, q_col=P, ld_q_col=16, s_col=P, scale=None, amax=None, nonfinite=None, stream=0)
    a.update(kw)
    return fm.fp8_rms_norm_quantize(**a)


@pytest.mark.parametrize("kw,code", [
    (dict(x_dtype=2), fm.ERR_ENUM), (dict(recipe=9), fm.ERR_ENUM), (dict(fmt=2), fm.ERR_ENUM), (dict(orient=0), fm.ERR_ENUM),
    (dict(recipe=fm.TENSOR_CURRENT), fm.ERR_UNSUPPORTED), (dict(recipe=fm.TENSOR_DELAYED, amax=P), fm.ERR_NULL),
    (dict(recipe=fm.TENSOR_DELAYED, scale=P), fm.ERR_NULL), (dict(recipe=fm.TENSOR_DELAYED, scale=P, amax=P + 2), fm.ERR_ALIGN),
    (dict(recipe=fm.TENSOR_DELAYED, scale=P + 1, amax=P), fm.ERR_ALIGN), (dict(recipe=fm.BLOCK_128x128), fm.ERR_UNSUPPORTED), (dict(recipe=fm.CHANNEL), fm.ERR_UNSUPPORTED), (dict(margin=65), fm.ERR_SHAPE),
    (dict(margin=-1), fm.ERR_SHAPE), (dict(eps=-1.0), fm.ERR_SHAPE), (dict(rows=-1), fm.ERR_SHAPE), (dict(x=None), fm.ERR_NULL),
    (dict(total=None), fm.ERR_NULL), (dict(rstd=None), fm.ERR_NULL), (dict(q_row=None), fm.ERR_NULL), (dict(s_row=None), fm.ERR_NULL),
    (dict(q_col=None), fm.ERR_NULL), (dict(s_col=None), fm.ERR_NULL), (dict(ld_q_row=48), fm.ERR_SHAPE),
    (dict(rows=17, ld_q_col=16), fm.ERR_SHAPE), (dict(ld_q_row=72), fm.ERR_ALIGN), (dict(ld_q_col=24), fm.ERR_ALIGN),
    (dict(q_row=P + 8), fm.ERR_ALIGN), (dict(q_col=P + 8), fm.ERR_ALIGN), (dict(s_row=P + 2), fm.ERR_ALIGN), (dict(s_col=P + 1), fm.ERR_ALIGN),
    (dict(nonfinite=P + 2), fm.ERR_ALIGN), (dict(ld_q_row=BIG), fm.ERR_SHAPE), (dict(rows=0), fm.OK),
])
def test_rms_quantize(kw, code):
    assert _quant(**kw) == code


def _back(**kw):
    a = dict(dy=P, ld_dy=64, total=P, x_dtype=fm.IN_BF16, rows=8, cols=64, ld_total=64, weight=P, w_dtype=fm.IN_FP32, rstd=P, dtotal=P,
             ld_dtotal=64, dx=P, ld_dx=64, dweight=P, workspace=P, workspace_bytes=1 << 20, stream=0)
    a.update(kw)
    return fm.fp8_rms_norm_backward(**a)


@pytest.mark.parametrize("kw,code", [
    (dict(x_dtype=2), fm.ERR_ENUM), (dict(cols=0), fm.ERR_SHAPE), (dict(dy=None), fm.ERR_NULL), (dict(total=None), fm.ERR_NULL),
    (dict(dx=None), fm.ERR_NULL), (dict(rstd=None), fm.ERR_NULL), (dict(workspace=None), fm.ERR_NULL), (dict(workspace_bytes=0), fm.ERR_SHAPE),
    (dict(ld_dy=1), fm.ERR_SHAPE), (dict(ld_dx=63), fm.ERR_SHAPE), (dict(ld_dtotal=63), fm.ERR_SHAPE), (dict(dy=P + 1), fm.ERR_ALIGN),
    (dict(dtotal=P + 1), fm.ERR_ALIGN), (dict(dweight=P + 1), fm.ERR_ALIGN), (dict(workspace=P + 2), fm.ERR_ALIGN),
    (dict(rows=0, dweight=None, workspace=None, dy=None, total=None, dx=None), fm.OK),
])
def test_rms_backward(kw, code):
    assert _back(**kw) == code


def test_sizes():
    assert fm.fp8_rms_norm_workspace(8, 64) >= 64 * 4 and fm.fp8_rms_norm_workspace(0, 64) > 0
    assert fm.fp8_rms_norm_workspace(-1, 64) == fm.fp8_rms_norm_workspace(8, 0) == fm.ERR_SHAPE
    assert fm.fp8_rms_norm_workspace(8, (1 << 28) + 1) == fm.ERR_UNSUPPORTED
    assert fm.fp8_moe_route_workspace(0, 8) == 0 and fm.fp8_moe_route_workspace(1000, 8) > 0 and fm.fp8_moe_route_workspace(1 << 20, 1024) > 0
    assert fm.fp8_moe_route_workspace(-1, 8) == fm.fp8_moe_route_workspace(8, 0) == fm.ERR_SHAPE
    assert fm.fp8_moe_route_workspace(1, 1025) == fm.fp8_moe_route_workspace((1 << 30) + 1, 8) == fm.ERR_UNSUPPORTED


def _route(**kw):
    a = dict(logits=P, dtype=fm.IN_FP32, tokens=1000, experts=8, ld_logits=8, mask=P, topk=2, normalize=1, expert=P, weights=P, loss=P,
             counts=P, slope=P, workspace=P, workspace_bytes=1 << 20, stream=0)
    a.update(kw)
    return fm.fp8_moe_route(**a)


ROUTE = [
    (dict(dtype=2), fm.ERR_ENUM), (dict(tokens=-1), fm.ERR_SHAPE), (dict(experts=0), fm.ERR_SHAPE), (dict(topk=0), fm.ERR_SHAPE),
    (dict(experts=1025, ld_logits=2000), fm.ERR_UNSUPPORTED), (dict(tokens=1 << 30), fm.ERR_UNSUPPORTED), (dict(tokens=BIG), fm.ERR_UNSUPPORTED),
    (dict(loss=None), fm.ERR_NULL), (dict(counts=None), fm.ERR_NULL), (dict(slope=None), fm.ERR_NULL), (dict(workspace=None), fm.ERR_NULL),
    (dict(workspace_bytes=16), fm.ERR_SHAPE), (dict(logits=None), fm.ERR_NULL), (dict(expert=None), fm.ERR_NULL),
    (dict(ld_logits=7), fm.ERR_SHAPE), (dict(ld_logits=BIG), fm.ERR_SHAPE), (dict(logits=P + 2), fm.ERR_ALIGN), (dict(expert=P + 2), fm.ERR_ALIGN),
    (dict(loss=P + 2), fm.ERR_ALIGN), (dict(workspace=P + 1), fm.ERR_ALIGN), (dict(counts=P + 1), fm.ERR_ALIGN),
]


@pytest.mark.parametrize("kw,code", ROUTE + [(dict(topk=9), fm.ERR_SHAPE), (dict(weights=None), fm.ERR_NULL), (dict(weights=P + 1), fm.ERR_ALIGN)])
def test_route(kw, code):
    assert _route(**kw) == code


@pytest.mark.parametrize("kw,code", ROUTE + [(dict(idx_dtype=2), fm.ERR_ENUM), (dict(ld_expert=1), fm.ERR_SHAPE),
                                             (dict(expert=P + 4, idx_dtype=fm.IDX_I64), fm.ERR_ALIGN)])
def test_balance(kw, code):
    a = dict(logits=P, dtype=fm.IN_FP32, tokens=1000, experts=8, ld_logits=8, mask=P, expert=P, idx_dtype=fm.IDX_I32, topk=2, ld_expert=2,
             loss=P, counts=P, slope=P, workspace=P, workspace_bytes=1 << 20, stream=0)
    a.update(kw)
    assert fm.fp8_moe_balance(**a) == code


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=2), fm.ERR_ENUM), (dict(tokens=-1), fm.ERR_SHAPE), (dict(topk=0), fm.ERR_SHAPE), (dict(topk=9), fm.ERR_SHAPE),
    (dict(experts=1025), fm.ERR_UNSUPPORTED), (dict(logits=None), fm.ERR_NULL), (dict(dlogits=None), fm.ERR_NULL), (dict(expert=None), fm.ERR_NULL), (dict(slope=None), fm.ERR_NULL),
    (dict(ld_logits=7), fm.ERR_SHAPE), (dict(ld_dlogits=7), fm.ERR_SHAPE), (dict(dlogits=P + 2), fm.ERR_ALIGN), (dict(dloss=P + 2), fm.ERR_ALIGN),
    (dict(expert=P + 2), fm.ERR_ALIGN), (dict(dweights=P + 1), fm.ERR_ALIGN), (dict(slope=P + 1), fm.ERR_ALIGN), (dict(tokens=0, logits=None), fm.OK),
])
def test_route_backward(kw, code):
    a = dict(logits=P, dtype=fm.IN_FP32, tokens=100, experts=8, ld_logits=8, mask=P, expert=P, topk=2, dweights=P, normalize=1, slope=P, dloss=P,
             dlogits=P, ld_dlogits=8, stream=0)
    a.update(kw)
    assert fm.fp8_moe_route_backward(**a) == code


def test_bindings_refuse_host_tensors():
    x, l = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(4, 8)
    s, e = torch.ones(8), torch.zeros(4, 2, dtype=torch.int32)
    for bad in (lambda: norm.rms_norm_forward(x), lambda: norm.rms_norm_quantize(x, fm.BLOCK_1x128, fm.E4M3),
                lambda: norm.rms_norm_backward(x, x, None, s), lambda: norm.RMSNorm(64)(x), lambda: moe.route(l, 2),
                lambda: moe.balance(l, e), lambda: moe.route_backward(l, e, l[:, :2], s, s),
                lambda: linear.RMSNormLinear(64, 64, recipe=linear.Float8BlockScaling())(x)):
        with pytest.raises(fm.Fp8Error, match="device tensor|GPU only"):
            bad()


def test_forward_mode_is_refused():
    from torch.autograd import forward_ad

    with forward_ad.dual_level():
        dual = forward_ad.make_dual(torch.zeros(4, 8), torch.ones(4, 8))
        with pytest.raises(fm.Fp8Error, match="forward-mode"):
            moe._wants_grad(dual)
