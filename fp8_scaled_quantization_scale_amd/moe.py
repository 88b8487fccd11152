"""Experts over the libfp8mi C ABI: tokens sorted by expert and back, and the
experts' scaled FP8 products on the sorted rows.

    plan = moe.sort(expert, experts)              # expert: [tokens x topk] from the router
    h = up(x, plan, gather=True)                  # GroupedLinear: dispatch, cast and products
    y = moe.combine(down(act(h), plan), plan, weights)

The sorted buffers have ``plan.rows`` rows, the most that any routing needs;
expert e's segment starts at ``plan.offsets[e]``, a multiple of 128, and ends
with rows of zeros.  The rows behind the last segment are never read or
written.  All sizes stay on the device: nothing here waits for the GPU, so a
step can be captured in a graph and replayed with other routings.
"""
from __future__ import annotations

from typing import NamedTuple

import torch
from torch.autograd import forward_ad
from torch.autograd.function import once_differentiable

from . import (BLOCK_1x128, COL, GEMM_MX_1x32, GROUP_CONTRACT, GROUP_ROWS, IDX_I32, IDX_I64, IN_BF16, IN_FP32,
               MAX_EXPERTS, MX_1x32, MX_1x32_OCP, OUT_BF16, OUT_FP32, ROW, Fp8Error, Quantized, _at, _ceil, _check, _dense, _here, _is_matrix,
               _is_vector, _ld, _matrix, _need, _one_device, _pad16, _scope, _vector, load, scale_grid_shape)
from . import quantize as _quantize_matrix

_DTYPES = {torch.bfloat16: IN_BF16, torch.float32: IN_FP32}
_OUT_DTYPES = {torch.bfloat16: OUT_BF16, torch.float32: OUT_FP32}
_IDX = {torch.int32: IDX_I32, torch.int64: IDX_I64}
_MOST_LD = 1 << 22  # leading dimension of a product's operands
_RECIPES = (BLOCK_1x128, MX_1x32, MX_1x32_OCP)
_CODES = (torch.uint8, torch.float8_e4m3fn, torch.float8_e5m2)


class _Fields(NamedTuple):
    tokens: int
    topk: int
    experts: int
    rows: int                # of the sorted buffers
    offsets: torch.Tensor    # [experts + 1] first row of each segment, and the end of the last
    counts: torch.Tensor     # [experts] slots of each
    row_slot: torch.Tensor   # [rows] slot (token * topk + choice) in each row, -1 where there is none
    slot_row: torch.Tensor   # [tokens x topk] row of each slot, -1 where it was dropped


class Plan(_Fields):
    """A routing's segments and row maps (int32 device tensors).  It cannot be
    changed, so its tensors' sizes are looked at once, here."""
    __slots__ = ()

    def __new__(cls, tokens, topk, experts, rows, offsets, counts, row_slot, slot_row):
        for name, t, n in (("offsets", offsets, experts + 1), ("counts", counts, experts), ("row_slot", row_slot, rows),
                           ("slot_row", slot_row, tokens * topk)):
            if not _is_vector(t, torch.int32, n):
                _vector("a plan's " + name, t, torch.int32, n)
        _one_device(offsets, counts, row_slot, slot_row)
        return super().__new__(cls, tokens, topk, experts, rows, offsets, counts, row_slot, slot_row)


def sort(expert: torch.Tensor, experts: int, stream=None) -> Plan:
    """Sort the slots of ``expert`` [tokens x topk] (int32 or int64) by expert,
    stably; numbers outside [0, experts) drop their slot."""
    if not _is_matrix(expert, _IDX):
        raise Fp8Error("expert must be a 2-D int32 or int64 device tensor with unit column stride")
    tokens, topk = expert.shape
    if topk < 1:
        raise Fp8Error("expert needs at least one choice per token")
    lib = load()  # (raises if the library is not built)
    rows = lib.fp8_moe_rows(tokens, topk, experts)
    if rows < 0:
        _check(rows, "fp8_moe_rows")
    size = lib.fp8_moe_sort_workspace(tokens, topk, experts)
    dev, i32 = expert.device, torch.int32
    with _scope(dev, stream):
        offsets, counts = torch.empty(experts + 1, dtype=i32, device=dev), torch.empty(experts, dtype=i32, device=dev)
        row_slot, slot_row = torch.empty(rows, dtype=i32, device=dev), torch.empty(tokens, topk, dtype=i32, device=dev)
        ws = torch.empty(size, dtype=torch.uint8, device=dev) if size else None
        st = lib.fp8_moe_sort(expert.data_ptr(), _IDX[expert.dtype], tokens, topk, _ld(expert), experts,
                              offsets.data_ptr(), counts.data_ptr(), row_slot.data_ptr(), rows, slot_row.data_ptr(),
                              _at(ws), size, _here(dev))
    _check(st, "fp8_moe_sort")
    return tuple.__new__(Plan, (tokens, topk, experts, rows, offsets, counts, row_slot, slot_row))


def _check_weights(p: Plan, weights) -> None:
    if weights is not None:
        n = p.tokens * p.topk
        if not _is_vector(weights, torch.float32, n):
            _vector("weights", weights, torch.float32, n)
        if weights.numel() != n:
            raise Fp8Error(f"weights is {tuple(weights.shape)}; needs {p.tokens} x {p.topk}")


def _rows_matrix(name: str, t: torch.Tensor, rows: int) -> None:
    if not _is_matrix(t, _DTYPES):
        _matrix(name, t, tuple(_DTYPES))
    if t.shape[0] != rows:
        raise Fp8Error(f"{name} has {t.shape[0]} rows; needs {rows}")


# ---------------------------------------------------------------------------
# rows to the experts and back
# ---------------------------------------------------------------------------

def _dispatch(x, plan, weights, stream):
    _rows_matrix("x", x, plan.tokens)
    _check_weights(plan, weights)
    _one_device(x, plan.slot_row, weights)
    cols = x.shape[1]
    with _scope(x.device, stream):
        y = torch.empty(plan.rows, cols, dtype=x.dtype, device=x.device)
        st = load().fp8_moe_dispatch(x.data_ptr(), _DTYPES[x.dtype], plan.tokens, cols, _ld(x), plan.topk, _at(weights),
                                     plan.slot_row.data_ptr(), plan.offsets.data_ptr(), plan.counts.data_ptr(),
                                     plan.experts, y.data_ptr(), plan.rows, cols, _here(x.device))
    _check(st, "fp8_moe_dispatch")
    return y


def _combine(ys, plan, weights, stream):
    _rows_matrix("ys", ys, plan.rows)
    _check_weights(plan, weights)
    _one_device(ys, plan.slot_row, weights)
    cols = ys.shape[1]
    with _scope(ys.device, stream):
        y = torch.empty(plan.tokens, cols, dtype=ys.dtype, device=ys.device)
        st = load().fp8_moe_combine(ys.data_ptr(), _DTYPES[ys.dtype], plan.rows, cols, _ld(ys), plan.slot_row.data_ptr(),
                                    plan.tokens, plan.topk, _at(weights), y.data_ptr(), cols, _here(ys.device))
    _check(st, "fp8_moe_combine")
    return y


def combine_backward(dy: torch.Tensor, ys: torch.Tensor | None, plan: Plan, weights: torch.Tensor | None,
                     rows: bool = True, dots: bool = True, stream=None):
    """The gradient of combine: (dys [plan.rows x cols] with zeros in the rows
    without a slot, dweights [tokens x topk] FP32).  rows=False or dots=False
    leaves one out (None); without dots, ys is not read and may be None."""
    _rows_matrix("dy", dy, plan.tokens)
    _check_weights(plan, weights)
    if dots:
        _rows_matrix("ys", ys, plan.rows)
        if ys.dtype != dy.dtype or ys.shape[1] != dy.shape[1]:
            raise Fp8Error("dy and ys must have one dtype and width")
    _one_device(dy, ys, plan.slot_row, weights)
    cols, dev = dy.shape[1], dy.device
    with _scope(dev, stream):
        dys = torch.empty(plan.rows, cols, dtype=dy.dtype, device=dev) if rows else None
        dw = torch.empty(plan.tokens, plan.topk, dtype=torch.float32, device=dev) if dots else None
        st = load().fp8_moe_combine_backward(dy.data_ptr(), _DTYPES[dy.dtype], plan.tokens, cols, _ld(dy),
                                             ys.data_ptr() if dots else None, _ld(ys) if dots else 0,
                                             plan.slot_row.data_ptr(), plan.offsets.data_ptr(), plan.counts.data_ptr(),
                                             plan.experts, plan.topk, _at(weights), _at(dys), plan.rows, cols, _at(dw),
                                             _here(dev))
    _check(st, "fp8_moe_combine_backward")
    return dys, dw


def _row_major(t: torch.Tensor) -> torch.Tensor:
    return t if t.stride(1) == 1 and _ld(t) >= t.shape[1] else _dense(t)


class _DispatchFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weights, plan):
        ctx.plan = plan
        ctx.save_for_backward(x if weights is not None else None, weights)
        return _dispatch(x, plan, weights, None)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        x, weights = ctx.saved_tensors
        dy, dx, dw = _row_major(dy), None, None
        if ctx.needs_input_grad[0]:
            dx = _combine(dy, ctx.plan, weights, None)
        if ctx.needs_input_grad[1]:
            dw = combine_backward(x, dy, ctx.plan, None, rows=False)[1].view(weights.shape)
        return dx, dw, None


class _CombineFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, ys, weights, plan):
        ctx.plan = plan
        ctx.save_for_backward(ys if weights is not None else None, weights)
        return _combine(ys, plan, weights, None)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        ys, weights = ctx.saved_tensors
        dys, dw = combine_backward(_row_major(dy), ys, ctx.plan, weights, ctx.needs_input_grad[0],
                                   ctx.needs_input_grad[1])
        return dys, None if dw is None else dw.view(weights.shape), None


def _wants_grad(*tensors) -> bool:
    for t in tensors:  # (a dual tensor need not require grad: its tangent would be lost without a word)
        if isinstance(t, torch.Tensor) and forward_ad.unpack_dual(t).tangent is not None:
            raise Fp8Error("dispatch and combine have no forward-mode derivative")
    return torch.is_grad_enabled() and any(t is not None and t.requires_grad for t in tensors)


def dispatch(x: torch.Tensor, plan: Plan, weights: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """The sorted rows [plan.rows x cols] of x [tokens x cols], each times its
    slot's weight.  Differentiable in x and weights, once and in reverse mode (on
    the current stream)."""
    if _wants_grad(x, weights):
        _need(stream is None, "with gradients, a call runs on the current stream")
        return _DispatchFn.apply(x, weights, plan)
    return _dispatch(x, plan, weights, stream)


def combine(ys: torch.Tensor, plan: Plan, weights: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Each token's sum [tokens x cols] of its slots' rows of ys [plan.rows x
    cols] times their weights (float [tokens x topk]; None: 1).  Differentiable
    in ys and weights, once and in reverse mode (on the current stream)."""
    if _wants_grad(ys, weights):
        _need(stream is None, "with gradients, a call runs on the current stream")
        return _CombineFn.apply(ys, weights, plan)
    return _combine(ys, plan, weights, stream)


def quantize(x: torch.Tensor, plan: Plan, recipe: int, fmt: int, orient: int = ROW, margin: int = 0,
             weights: torch.Tensor | None = None, gather: bool = True, nonfinite: torch.Tensor | None = None,
             stream=None) -> Quantized:
    """FP8 codes and scales of the sorted rows: of x [tokens x cols] read through
    the plan (gather), each row times its slot's weight, or of x [plan.rows x
    cols] itself.  recipe: BLOCK_1x128, MX_1x32 or MX_1x32_OCP."""
    _rows_matrix("x", x, plan.tokens if gather else plan.rows)
    _check_weights(plan, weights)
    if nonfinite is not None:
        _vector("nonfinite", nonfinite, torch.int32, 1)
    _one_device(x, plan.offsets, weights, nonfinite)
    if recipe not in _RECIPES:
        raise Fp8Error("experts take the recipes BLOCK_1x128, MX_1x32 and MX_1x32_OCP: other scales would span experts")
    rows, cols, dev = plan.rows, x.shape[1], x.device
    out = Quantized(fmt=fmt, recipe=recipe, nonfinite=nonfinite)
    ld_r, ld_c = _pad16(cols), rows  # (rows: a multiple of 128, or none, which a product takes as its contraction)
    with _scope(dev, stream):
        if orient & ROW:
            out.q_row = torch.empty(rows, ld_r, dtype=torch.uint8, device=dev)
            shp, dt = scale_grid_shape(recipe, rows, cols, ROW)
            out.s_row = torch.empty(shp, dtype=dt, device=dev)
        if orient & COL:
            out.q_col = torch.empty(cols, ld_c, dtype=torch.uint8, device=dev)
            shp, dt = scale_grid_shape(recipe, rows, cols, COL)
            out.s_col = torch.empty(shp, dtype=dt, device=dev)
        st = load().fp8_moe_quantize(x.data_ptr(), _DTYPES[x.dtype], x.shape[0], cols, _ld(x),
                                     plan.row_slot.data_ptr() if gather else None, plan.topk, _at(weights),
                                     plan.offsets.data_ptr(), plan.experts, rows, recipe, fmt, orient, margin,
                                     _at(out.q_row), ld_r, _at(out.s_row), _at(out.q_col), ld_c, _at(out.s_col),
                                     _at(nonfinite), _here(dev))
    _check(st, "fp8_moe_quantize")
    return out


# ---------------------------------------------------------------------------
# the experts' products
# ---------------------------------------------------------------------------

def _offsets(offsets: torch.Tensor) -> int:
    if not (_is_vector(offsets, torch.int32, 2) and offsets.dim() == 1):
        raise Fp8Error("offsets must be a contiguous int32 device vector of experts + 1 numbers")
    return offsets.numel() - 1


def _out_of(c, shape, out_dtype, device) -> torch.Tensor:
    if c is None:
        if out_dtype not in _OUT_DTYPES:
            raise Fp8Error(f"out_dtype must be one of {tuple(_OUT_DTYPES)}")
        return torch.empty(shape, dtype=out_dtype, device=device)
    if not (isinstance(c, torch.Tensor) and c.is_cuda and c.dtype in _OUT_DTYPES and tuple(c.shape) == shape
            and (c.stride(-1) == 1 or shape[-1] <= 1)):
        raise Fp8Error(f"c must be a BF16 or FP32 device tensor {shape} with unit last stride")
    return c


def gemm(a: torch.Tensor, fmt_a: int, s_a: torch.Tensor, b: torch.Tensor, fmt_b: int, s_b: torch.Tensor, recipe: int,
         offsets: torch.Tensor, out_dtype=torch.bfloat16, c: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """c[r] = dequant(a[r, :K]) . dequant(b[e])^T for the rows r of segment e.

    a [rows x >= K] codes with their scales [rows x blocks]; b [experts x N x K]
    codes and s_b [experts x N/128 x K/128] tile scales (GEMM_MX_1x32: [experts
    x N x K/32] bytes), each with unit last stride and any others, so that a
    view of transposed codes will do.  Rows behind the last segment are left as
    they were."""
    if not _is_matrix(a, _CODES):
        _matrix("a", a, _CODES)
    experts = _offsets(offsets)
    if not (isinstance(b, torch.Tensor) and b.is_cuda and b.dtype in _CODES and b.dim() == 3 and b.shape[0] == experts
            and (b.stride(2) == 1 or b.shape[2] <= 1)):
        raise Fp8Error(f"b must be a device tensor of codes, {experts} x N x K with unit last stride")
    rows, (_, n, k) = a.shape[0], b.shape
    if a.shape[1] < k:
        raise Fp8Error(f"a is {tuple(a.shape)}; needs at least {rows} x {k}")
    mx = recipe == GEMM_MX_1x32
    dtype = torch.uint8 if mx else torch.float32
    grid = (experts, n if mx else _ceil(n, 128), _ceil(k, 32 if mx else 128))
    if not _is_vector(s_a, dtype, rows * grid[2]):
        _vector("s_a", s_a, dtype, rows * grid[2])
    if not (isinstance(s_b, torch.Tensor) and s_b.is_cuda and s_b.dtype == dtype and tuple(s_b.shape) == grid
            and (s_b.stride(2) == 1 or grid[2] <= 1)):
        raise Fp8Error(f"s_b must be a {dtype} device tensor {grid} with unit last stride")
    _one_device(a, offsets, s_a, b, s_b, c)
    with _scope(a.device, stream):
        c = _out_of(c, (rows, n), out_dtype, a.device)
        st = load().fp8_gemm_grouped(a.data_ptr(), fmt_a, s_a.data_ptr(), _ld(a), b.data_ptr(), fmt_b, s_b.data_ptr(),
                                     b.stride(1) if n > 1 else max(b.stride(1), k), b.stride(0) if experts > 1 else 0,
                                     s_b.stride(1) if grid[1] > 1 else max(s_b.stride(1), grid[2]),
                                     s_b.stride(0) if experts > 1 else 0, recipe, GROUP_ROWS, offsets.data_ptr(),
                                     experts, rows, 0, n, k, c.data_ptr(), _OUT_DTYPES[c.dtype], _ld(c), 0,
                                     _here(a.device))
    _check(st, "fp8_gemm_grouped")
    return c


def gemm_wgrad(a: torch.Tensor, fmt_a: int, s_a: torch.Tensor, b: torch.Tensor, fmt_b: int, s_b: torch.Tensor,
               recipe: int, offsets: torch.Tensor, out_dtype=torch.bfloat16, c: torch.Tensor | None = None,
               stream=None) -> torch.Tensor:
    """c[e] = dequant(a[:, segment e]) . dequant(b[:, segment e])^T for every
    expert: a [M x rows], b [N x rows] the transposed codes of the sorted rows
    (quantize's COL outputs), s_a and s_b their grids [M x rows/128] and [N x
    rows/128] (GEMM_MX_1x32: rows/32 bytes); c [experts x M x N] with unit last
    stride, the experts one after the other or their rows in turn."""
    for name, t in (("a", a), ("b", b)):
        if not _is_matrix(t, _CODES):
            _matrix(name, t, _CODES)
    experts = _offsets(offsets)
    (m, rows), n = a.shape, b.shape[0]
    if b.shape[1] != rows:
        raise Fp8Error(f"a has {rows} columns, b {b.shape[1]}")
    mx = recipe == GEMM_MX_1x32
    dtype = torch.uint8 if mx else torch.float32
    for name, t, size in (("s_a", s_a, m * _ceil(rows, 32 if mx else 128)), ("s_b", s_b, n * _ceil(rows, 32 if mx else 128))):
        if not _is_vector(t, dtype, size):
            _vector(name, t, dtype, size)
    _one_device(a, offsets, s_a, b, s_b, c)
    with _scope(a.device, stream):
        c = _out_of(c, (experts, m, n), out_dtype, a.device)
        ldc = c.stride(1) if m > 1 else max(c.stride(1), n)
        st = load().fp8_gemm_grouped(a.data_ptr(), fmt_a, s_a.data_ptr(), _ld(a), b.data_ptr(), fmt_b, s_b.data_ptr(),
                                     _ld(b), 0, 0, 0, recipe, GROUP_CONTRACT, offsets.data_ptr(), experts, rows, m, n,
                                     0, c.data_ptr(), _OUT_DTYPES[c.dtype], ldc, c.stride(0), _here(a.device))
    _check(st, "fp8_gemm_grouped")
    return c


# ---------------------------------------------------------------------------
# the layer
# ---------------------------------------------------------------------------

def _out(dtype):
    return torch.float32 if dtype == torch.float32 else torch.bfloat16


class _GroupedLinearFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, mplan, p, gather, need_dx, need_dw):
        e, n, k = weight.shape
        (rx, fx), (rw, fw) = p.quant["x"], p.quant["w"]
        qx = quantize(x, mplan, rx, fx, ROW | (COL if need_dw else 0), gather=gather)
        # all experts' weights as one matrix: with whole blocks per expert its
        # transposed codes are the experts' transposed codes side by side
        qw = _quantize_matrix(weight.reshape(e * n, k), rw, fw, ROW | (COL if need_dx else 0))
        y = gemm(qx.q_row, fx, qx.s_row, qw.q_row.view(e, n, -1), fw, qw.s_row.view(e, -1, qw.s_row.shape[1]),
                 p.gemm["fprop"], mplan.offsets, _out(x.dtype))
        ctx.p, ctx.mplan, ctx.gather, ctx.need = p, mplan, gather, (need_dx, need_dw)
        ctx.shape, ctx.dtypes = (e, n, k), (x.dtype, weight.dtype)
        ctx.save_for_backward(*((qx.q_col, qx.s_col) if need_dw else (None, None)),
                              *((qw.q_col, qw.s_col) if need_dx else (None, None)))
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        qxt, sxt, qwt, swt = ctx.saved_tensors
        p, mplan, (e, n, k), (need_dx, need_dw) = ctx.p, ctx.mplan, ctx.shape, ctx.need
        (_, fx), (_, fw), (rg, fg) = p.quant["x"], p.quant["w"], p.quant["g"]
        dy = _dense(dy)
        if dy.dtype not in _DTYPES:
            dy = dy.float()
        qg = quantize(dy, mplan, rg, fg, (ROW if need_dx else 0) | (COL if need_dw else 0), gather=False)
        dx = dw = None
        if need_dx:
            dx = gemm(qg.q_row, fg, qg.s_row, qwt.view(k, e, n).permute(1, 0, 2), fw,
                      swt.view(swt.shape[0], e, -1).permute(1, 0, 2), p.gemm["dgrad"], mplan.offsets,
                      _out(ctx.dtypes[0]))
            if ctx.gather:
                dx = _combine(dx, mplan, None, None)
        if need_dw:
            dw = gemm_wgrad(qg.q_col, fg, qg.s_col, qxt, fx, sxt, p.gemm["wgrad"], mplan.offsets, _out(ctx.dtypes[1]))
        return dx, dw, None, None, None, None, None


class GroupedLinear(torch.nn.Module):
    """One weight [out_features x in_features] per expert, y[r] = x[r] W_e^T on
    sorted rows, with FP8 products in both passes; the recipes are those of
    ``linear.Linear`` whose scales stay inside a row or a block
    (Float8BlockScaling and MXFP8BlockScaling).

    ``forward(x, plan)`` takes the sorted rows [plan.rows x in_features], with
    zeros in a segment's rows without a slot (as dispatch, combine's gradient
    and this layer itself leave them); ``gather=True`` takes x [tokens x
    in_features] and dispatches it as it is cast.  in_features and out_features
    are multiples of 128, so that no block holds two experts' weights; experts *
    out_features is at most 4194304, and so are plan.rows where the weight needs
    a gradient (the leading dimensions that the products take)."""

    def __init__(self, experts: int, in_features: int, out_features: int, recipe=None, device=None,
                 dtype=torch.bfloat16):
        super().__init__()
        if experts < 1 or in_features < 128 or out_features < 128 or in_features % 128 or out_features % 128:
            raise Fp8Error("experts must be positive, in_features and out_features multiples of 128")
        if experts > MAX_EXPERTS or experts * out_features > _MOST_LD or in_features > _MOST_LD:
            raise Fp8Error(f"at most {MAX_EXPERTS} experts, and at most {_MOST_LD} features in all")
        self.experts, self.in_features, self.out_features, self.recipe = experts, in_features, out_features, recipe
        self.weight = torch.nn.Parameter(torch.empty(experts, out_features, in_features, device=device, dtype=dtype))
        torch.nn.init.uniform_(self.weight, -in_features ** -0.5, in_features ** -0.5)

    def forward(self, x: torch.Tensor, plan: Plan, gather: bool = False) -> torch.Tensor:
        from . import linear

        r = linear.active_recipe() or self.recipe
        if r is None:
            raise Fp8Error("no FP8 recipe: pass recipe= or call inside fp8_autocast")
        p = linear.plan(r)
        if not isinstance(r, (linear.Float8BlockScaling, linear.MXFP8BlockScaling)):
            raise Fp8Error("experts take the block recipes only: other scales would span experts")
        if not x.is_cuda or not self.weight.is_cuda:
            raise Fp8Error("the grouped linear layer runs on the GPU only")
        if x.dim() != 2 or x.shape[1] != self.in_features:
            raise Fp8Error(f"input is {tuple(x.shape)}; needs {self.in_features} columns")
        if plan.experts != self.experts:
            raise Fp8Error(f"the plan has {plan.experts} experts, the layer {self.experts}")
        if x.dtype not in _DTYPES or self.weight.dtype not in _DTYPES:
            raise Fp8Error("inputs and weights are BF16 or FP32")
        grad = torch.is_grad_enabled()
        if grad and self.weight.requires_grad and plan.rows > _MOST_LD:
            raise Fp8Error(f"the weight's gradient takes at most {_MOST_LD} sorted rows; the plan has {plan.rows}")
        return _GroupedLinearFn.apply(_dense(x), self.weight.contiguous(), plan, p, gather,
                                      grad and x.requires_grad, grad and self.weight.requires_grad)
