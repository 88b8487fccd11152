"""The layer norm's and the experts' C entry points refuse bad arguments before
any GPU work (only invalid and empty calls are made), and the bindings refuse
host tensors."""
import pytest
import torch

import fp8_scaled_quantization_scale_amd as fm
from fp8_scaled_quantization_scale_amd import moe, norm

P = 0x10000  # an aligned stand-in pointer, never dereferenced
BIG = 1 << 62


def _norm(**kw):
    a = dict(x=P, x_dtype=fm.IN_BF16, rows=8, cols=64, ld_x=64, weight=P, bias=P, w_dtype=fm.IN_FP32, eps=1e-5, y=P, ld_y=64,
             mean=P, rstd=P, stream=0)
    a.update(kw)
    return fm.fp8_layer_norm_forward(**a)


@pytest.mark.parametrize("kw,code", [
    (dict(x_dtype=2), fm.ERR_ENUM), (dict(w_dtype=-1), fm.ERR_ENUM), (dict(rows=-1), fm.ERR_SHAPE), (dict(cols=0), fm.ERR_SHAPE),
    (dict(cols=(1 << 28) + 1, ld_x=BIG, ld_y=BIG), fm.ERR_UNSUPPORTED), (dict(eps=-1e-9), fm.ERR_SHAPE),
    (dict(eps=float("nan")), fm.ERR_SHAPE), (dict(x=None), fm.ERR_NULL), (dict(y=None), fm.ERR_NULL), (dict(mean=None), fm.ERR_NULL),
    (dict(rstd=None), fm.ERR_NULL), (dict(ld_x=63), fm.ERR_SHAPE), (dict(ld_y=63), fm.ERR_SHAPE), (dict(ld_x=BIG), fm.ERR_SHAPE),
    (dict(x=P + 1), fm.ERR_ALIGN), (dict(y=P + 1), fm.ERR_ALIGN), (dict(mean=P + 2), fm.ERR_ALIGN), (dict(weight=P + 2), fm.ERR_ALIGN),
    (dict(bias=P + 1), fm.ERR_ALIGN), (dict(x=P + 2, x_dtype=fm.IN_FP32), fm.ERR_ALIGN), (dict(rows=0, x=None, y=None), fm.OK),
])
def test_norm_forward(kw, code):
    assert _norm(**kw) == code


def _norm_b(**kw):
    a = dict(dy=P, ld_dy=64, x=P, x_dtype=fm.IN_BF16, rows=8, cols=64, ld_x=64, weight=P, w_dtype=fm.IN_FP32, mean=P, rstd=P, dx=P,
             ld_dx=64, dweight=P, dbias=P, workspace=P, workspace_bytes=1 << 20, stream=0)
    a.update(kw)
    return fm.fp8_layer_norm_backward(**a)


@pytest.mark.parametrize("kw,code", [
    (dict(x_dtype=2), fm.ERR_ENUM), (dict(cols=0), fm.ERR_SHAPE), (dict(dy=None), fm.ERR_NULL), (dict(x=None), fm.ERR_NULL),
    (dict(dx=None), fm.ERR_NULL), (dict(mean=None), fm.ERR_NULL), (dict(workspace=None), fm.ERR_NULL),
    (dict(workspace_bytes=0), fm.ERR_SHAPE), (dict(ld_dy=1), fm.ERR_SHAPE), (dict(ld_dx=63), fm.ERR_SHAPE),
    (dict(dy=P + 1), fm.ERR_ALIGN), (dict(dweight=P + 1), fm.ERR_ALIGN), (dict(workspace=P + 2), fm.ERR_ALIGN),
    (dict(rows=0, dweight=None, dbias=None, workspace=None, dy=None, x=None, dx=None), fm.OK),
])
def test_norm_backward(kw, code):
    assert _norm_b(**kw) == code


def test_sizes():
    assert fm.fp8_layer_norm_workspace(8, 64) >= 2 * 64 * 4 and fm.fp8_layer_norm_workspace(0, 64) > 0
    assert fm.fp8_layer_norm_workspace(-1, 64) == fm.fp8_layer_norm_workspace(8, 0) == fm.ERR_SHAPE
    assert fm.fp8_moe_rows(0, 2, 8) == 0 and fm.fp8_moe_rows(1, 1, 1) == 128 and fm.fp8_moe_rows(128, 1, 1) == 128
    assert fm.fp8_moe_rows(64, 2, 1) == 128 and fm.fp8_moe_rows(1, 2, 100) == 256
    assert fm.fp8_moe_rows(-1, 2, 8) == fm.fp8_moe_rows(1, 0, 8) == fm.fp8_moe_rows(1, 1, 0) == fm.ERR_SHAPE
    for bad in ((1, 1, 1025), (1 << 31, 1, 1), (1 << 29, 4, 1), (1, 1 << 31, 1), (BIG, BIG, 1)):
        assert fm.fp8_moe_rows(*bad) == fm.fp8_moe_sort_workspace(*bad) == fm.ERR_UNSUPPORTED
    assert fm.fp8_moe_sort_workspace(100, 2, 8) == 0 and fm.fp8_moe_sort_workspace(1 << 20, 8, 256) > 0


def _sort(**kw):
    a = dict(expert=P, idx_dtype=fm.IDX_I64, tokens=100, topk=2, ld_expert=2, experts=8, offsets=P, counts=P, row_slot=P, rows=1152,
             slot_row=P, workspace=None, workspace_bytes=0, stream=0)
    a.update(kw)
    return fm.fp8_moe_sort(**a)


@pytest.mark.parametrize("kw,code", [
    (dict(idx_dtype=2), fm.ERR_ENUM), (dict(tokens=-1), fm.ERR_SHAPE), (dict(topk=0), fm.ERR_SHAPE), (dict(experts=0), fm.ERR_SHAPE),
    (dict(experts=1025), fm.ERR_UNSUPPORTED), (dict(tokens=1 << 30), fm.ERR_UNSUPPORTED), (dict(rows=1151), fm.ERR_SHAPE),
    (dict(rows=1024), fm.ERR_SHAPE), (dict(expert=None), fm.ERR_NULL), (dict(offsets=None), fm.ERR_NULL), (dict(counts=None), fm.ERR_NULL),
    (dict(row_slot=None), fm.ERR_NULL), (dict(slot_row=None), fm.ERR_NULL), (dict(ld_expert=1), fm.ERR_SHAPE),
    (dict(expert=P + 4), fm.ERR_ALIGN), (dict(offsets=P + 2), fm.ERR_ALIGN),
    (dict(tokens=10000, rows=1 << 20), fm.ERR_NULL),  # needs a workspace
    (dict(tokens=10000, rows=1 << 20, workspace=P), fm.ERR_SHAPE),
])
def test_sort(kw, code):
    assert fm.fp8_moe_rows(100, 2, 8) == 1152
    assert _sort(**kw) == code


def _dispatch(**kw):
    a = dict(x=P, dtype=fm.IN_BF16, tokens=100, cols=64, ld_x=64, topk=2, weights=P, slot_row=P, offsets=P, counts=P, experts=8, y=P,
             rows=1152, ld_y=64, stream=0)
    a.update(kw)
    return fm.fp8_moe_dispatch(**a)


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=3), fm.ERR_ENUM), (dict(rows=100), fm.ERR_SHAPE), (dict(cols=-1), fm.ERR_SHAPE), (dict(x=None), fm.ERR_NULL),
    (dict(y=None), fm.ERR_NULL), (dict(slot_row=None), fm.ERR_NULL), (dict(counts=None), fm.ERR_NULL), (dict(ld_x=63), fm.ERR_SHAPE),
    (dict(x=P + 1), fm.ERR_ALIGN), (dict(weights=P + 2), fm.ERR_ALIGN), (dict(tokens=1 << 28, cols=1 << 24, ld_x=1 << 24), fm.ERR_UNSUPPORTED),
    (dict(tokens=0, x=None), fm.OK), (dict(cols=0), fm.OK),
])
def test_dispatch(kw, code):
    assert _dispatch(**kw) == code


def _quantize(**kw):
    a = dict(x=P, x_dtype=fm.IN_BF16, x_rows=100, cols=64, ld_x=64, row_slot=P, topk=2, weights=P, offsets=P, experts=8, rows=1152,
             recipe=fm.BLOCK_1x128, fmt=fm.E4M3, orient=fm.ROW_AND_COL, margin=0, q_row=P, ld_q_row=64, s_row=P, q_col=P,
             ld_q_col=1152, s_col=P, nonfinite=None, stream=0)
    a.update(kw)
    return fm.fp8_moe_quantize(**a)


@pytest.mark.parametrize("kw,code", [
    (dict(x_dtype=2), fm.ERR_ENUM), (dict(recipe=9), fm.ERR_ENUM), (dict(fmt=2), fm.ERR_ENUM), (dict(orient=0), fm.ERR_ENUM),
    (dict(recipe=fm.TENSOR_CURRENT), fm.ERR_UNSUPPORTED), (dict(recipe=fm.BLOCK_128x128), fm.ERR_UNSUPPORTED),
    (dict(recipe=fm.CHANNEL), fm.ERR_UNSUPPORTED), (dict(margin=65), fm.ERR_SHAPE), (dict(rows=1100), fm.ERR_SHAPE),
    (dict(topk=0), fm.ERR_SHAPE), (dict(row_slot=None, weights=None), fm.ERR_SHAPE),  # x has too few rows to be read as they are
    (dict(row_slot=None, x_rows=1152), fm.ERR_SHAPE),  # weights need slots
    (dict(x=None), fm.ERR_NULL), (dict(offsets=None), fm.ERR_NULL), (dict(q_row=None), fm.ERR_NULL), (dict(s_col=None), fm.ERR_NULL),
    (dict(ld_x=56), fm.ERR_SHAPE), (dict(ld_q_col=1136), fm.ERR_SHAPE), (dict(ld_x=68), fm.ERR_ALIGN), (dict(q_row=P + 8), fm.ERR_ALIGN),
    (dict(rows=0), fm.OK), (dict(cols=0), fm.OK),
])
def test_quantize(kw, code):
    assert _quantize(**kw) == code


def _combine(**kw):
    a = dict(ys=P, dtype=fm.IN_BF16, rows=1152, cols=64, ld_ys=64, slot_row=P, tokens=100, topk=2, weights=P, y=P, ld_y=64, stream=0)
    a.update(kw)
    return fm.fp8_moe_combine(**a)


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=3), fm.ERR_ENUM), (dict(rows=-128), fm.ERR_SHAPE), (dict(ys=None), fm.ERR_NULL), (dict(y=None), fm.ERR_NULL),
    (dict(slot_row=None), fm.ERR_NULL), (dict(ld_ys=63), fm.ERR_SHAPE), (dict(ys=P + 1), fm.ERR_ALIGN), (dict(topk=0), fm.ERR_SHAPE),
    (dict(tokens=0, ys=None, y=None), fm.OK),
])
def test_combine(kw, code):
    assert _combine(**kw) == code


def _combine_b(**kw):
    a = dict(dy=P, dtype=fm.IN_BF16, tokens=100, cols=64, ld_dy=64, ys=P, ld_ys=64, slot_row=P, offsets=P, counts=P, experts=8, topk=2,
             weights=P, dys=P, rows=1152, ld_dys=64, dweights=P, stream=0)
    a.update(kw)
    return fm.fp8_moe_combine_backward(**a)


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=3), fm.ERR_ENUM), (dict(experts=0), fm.ERR_SHAPE), (dict(dy=None), fm.ERR_NULL), (dict(ys=None), fm.ERR_NULL),
    (dict(slot_row=None), fm.ERR_NULL), (dict(offsets=None), fm.ERR_NULL), (dict(ld_dys=63), fm.ERR_SHAPE),
    (dict(dweights=P + 2), fm.ERR_ALIGN), (dict(dys=None, dweights=None, dy=None), fm.OK), (dict(tokens=0), fm.OK),
])
def test_combine_backward(kw, code):
    assert _combine_b(**kw) == code


def _gemm(**kw):
    a = dict(a=P, fmt_a=fm.E4M3, s_a=P, lda=256, b=P, fmt_b=fm.E4M3, s_b=P, ldb=256, stride_b=256 * 128, ld_sb=2, stride_sb=2,
             recipe=fm.GEMM_BLOCK_1x128_128x128, group=fm.GROUP_ROWS, offsets=P, experts=8, rows=1152, M=0, N=128, K=256, c=P,
             c_dtype=fm.OUT_BF16, ldc=128, stride_c=0, stream=0)
    a.update(kw)
    return fm.fp8_gemm_grouped(**a)


CONTRACT = dict(group=fm.GROUP_CONTRACT, recipe=fm.GEMM_BLOCK_1x128_1x128, M=64, lda=1152, ldb=1152, stride_c=64 * 128)


@pytest.mark.parametrize("kw,code", [
    (dict(fmt_a=2), fm.ERR_ENUM), (dict(recipe=7), fm.ERR_ENUM), (dict(group=2), fm.ERR_ENUM), (dict(c_dtype=2), fm.ERR_ENUM),
    (dict(recipe=fm.GEMM_TENSOR), fm.ERR_UNSUPPORTED), (dict(recipe=fm.GEMM_BLOCK_1x128_1x128), fm.ERR_UNSUPPORTED),
    (dict(experts=0), fm.ERR_SHAPE), (dict(experts=1025), fm.ERR_UNSUPPORTED), (dict(rows=1000), fm.ERR_SHAPE), (dict(N=-1), fm.ERR_SHAPE),
    (dict(K=-16), fm.ERR_SHAPE), (dict(K=250), fm.ERR_SHAPE), (dict(c=None), fm.ERR_NULL), (dict(offsets=None), fm.ERR_NULL),
    (dict(a=None), fm.ERR_NULL), (dict(s_b=None), fm.ERR_NULL), (dict(lda=128), fm.ERR_SHAPE), (dict(ldb=264), fm.ERR_ALIGN),
    (dict(stride_b=8), fm.ERR_SHAPE), (dict(stride_b=-16), fm.ERR_SHAPE), (dict(ld_sb=1), fm.ERR_SHAPE), (dict(stride_sb=-1), fm.ERR_SHAPE),
    (dict(ld_sb=1 << 23), fm.ERR_UNSUPPORTED), (dict(lda=(1 << 22) + 16), fm.ERR_UNSUPPORTED), (dict(ldc=127), fm.ERR_SHAPE),
    (dict(a=P + 8), fm.ERR_ALIGN), (dict(s_a=P + 2), fm.ERR_ALIGN), (dict(offsets=P + 1), fm.ERR_ALIGN), (dict(c=P + 1), fm.ERR_ALIGN),
    (dict(rows=0), fm.OK), (dict(N=0, c=None), fm.OK),
    (dict(CONTRACT, recipe=fm.GEMM_BLOCK_1x128_128x128), fm.ERR_UNSUPPORTED), (dict(CONTRACT, M=-1), fm.ERR_SHAPE),
    (dict(CONTRACT, lda=1136), fm.ERR_SHAPE), (dict(CONTRACT, stride_c=-1), fm.ERR_SHAPE), (dict(CONTRACT, ldc=64), fm.ERR_SHAPE),
    (dict(CONTRACT, rows=1 << 23, lda=1 << 23, ldb=1 << 23), fm.ERR_UNSUPPORTED), (dict(CONTRACT, M=0), fm.OK),
    (dict(CONTRACT, experts=1024, M=1 << 30, N=1 << 30, ldc=1 << 30), fm.ERR_UNSUPPORTED),
])
def test_gemm_grouped(kw, code):
    assert _gemm(**kw) == code


def test_bindings_refuse_host_tensors():
    x, e = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(4, 2, dtype=torch.int64)
    i = torch.zeros(8, dtype=torch.int32)
    plan = tuple.__new__(moe.Plan, (4, 2, 7, 8, i, i, i, i))
    q, s = torch.zeros(128, 64, dtype=torch.uint8), torch.ones(128)
    for bad in (lambda: norm.layer_norm_forward(x), lambda: norm.layer_norm_backward(x, x, None, s, s), lambda: moe.sort(e, 8),
                lambda: moe.dispatch(x, plan), lambda: moe.combine(x, plan), lambda: moe.combine_backward(x, x, plan, None),
                lambda: moe.quantize(x, plan, fm.BLOCK_1x128, fm.E4M3),
                lambda: moe.gemm(q, 0, s, q.view(1, 128, 64), 0, s, fm.GEMM_MX_1x32, i), lambda: moe.gemm_wgrad(q, 0, s, q, 0, s, 3, i),
                lambda: moe.Plan(4, 2, 7, 8, i, i, i, i), lambda: norm.LayerNorm(64)(x)):
        with pytest.raises(fm.Fp8Error, match="device tensor|device vector|GPU only"):
            bad()
