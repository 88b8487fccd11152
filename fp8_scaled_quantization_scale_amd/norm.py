"""Layer norm and RMS norm over the libfp8mi C ABI: the layer before an FP8
linear layer.

``layer_norm_forward`` / ``layer_norm_backward`` and ``rms_norm_forward`` /
``rms_norm_quantize`` / ``rms_norm_backward`` allocate their outputs with torch
and call the entry points of include/fp8mi.h; ``LayerNorm`` and ``RMSNorm`` drive
them through autograd (and ``linear.RMSNormLinear`` the norm into FP8 codes with
the product that takes them).  BF16 or FP32 activations, BF16 or FP32 parameters,
FP32 statistics and sums.
"""
from __future__ import annotations

import torch
from torch.autograd.function import once_differentiable

from . import (AMAX_SLOTS, BLOCK_1x128, COL, IN_BF16, IN_FP32, MX_1x32, MX_1x32_OCP, ROW, TENSOR_DELAYED, Fp8Error, Quantized, _at, _check, _dense,
               _here, _is_matrix, _is_vector, _ld, _matrix, _one_device, _pad16, _scope, _vector, load, scale_grid_shape)

_DTYPES = {torch.bfloat16: IN_BF16, torch.float32: IN_FP32}


def _check_x(x) -> None:
    if not _is_matrix(x, _DTYPES):
        _matrix("x", x, tuple(_DTYPES))
    if x.shape[1] < 1:
        raise Fp8Error("x needs at least one column")


def _params(cols: int, weight, bias):
    """dtype of the parameters (FP32 where there are none)."""
    dtype = None
    for t in (weight, bias):
        if t is None:
            continue
        if not (isinstance(t, torch.Tensor) and t.is_cuda and t.dtype in _DTYPES and t.is_contiguous()):
            raise Fp8Error("weight and bias must be contiguous BF16 or FP32 device tensors")
        if t.dim() != 1 or t.numel() != cols or t.dtype != (dtype or t.dtype):
            raise Fp8Error(f"weight and bias must have one dtype and {cols} elements each")
        dtype = t.dtype
    return dtype or torch.float32


def layer_norm_forward(x: torch.Tensor, weight: torch.Tensor | None = None, bias: torch.Tensor | None = None,
                       eps: float = 1e-5, stream=None):
    """(y, mean, rstd) of the rows of a 2-D x (unit column stride): y as x, the
    FP32 statistics for layer_norm_backward."""
    _check_x(x)
    rows, cols = x.shape
    w_dtype = _params(cols, weight, bias)
    _one_device(x, weight, bias)
    dev = x.device
    with _scope(dev, stream):
        y = torch.empty(rows, cols, dtype=x.dtype, device=dev)
        mean = torch.empty(rows, dtype=torch.float32, device=dev)
        rstd = torch.empty(rows, dtype=torch.float32, device=dev)
        st = load().fp8_layer_norm_forward(x.data_ptr(), _DTYPES[x.dtype], rows, cols, _ld(x), _at(weight), _at(bias),
                                           _DTYPES[w_dtype], eps, y.data_ptr(), cols, mean.data_ptr(), rstd.data_ptr(),
                                           _here(dev))
    _check(st, "fp8_layer_norm_forward")
    return y, mean, rstd


def layer_norm_backward(dy: torch.Tensor, x: torch.Tensor, weight: torch.Tensor | None, mean: torch.Tensor,
                        rstd: torch.Tensor, params: bool = True, stream=None):
    """(dx, dweight, dbias); params=False leaves the last two out (None).  They
    take the weight's dtype, FP32 where there is no weight."""
    _check_x(x)
    if not _is_matrix(dy, (x.dtype,)):
        _matrix("dy", dy, (x.dtype,))
    rows, cols = x.shape
    if dy.shape != x.shape:
        raise Fp8Error(f"dy is {tuple(dy.shape)}, x {tuple(x.shape)}")
    w_dtype = _params(cols, weight, None)
    for name, t in (("mean", mean), ("rstd", rstd)):
        if not _is_vector(t, torch.float32, rows):
            _vector(name, t, torch.float32, rows)
    _one_device(x, dy, weight, mean, rstd)
    dev = x.device
    with _scope(dev, stream):
        dx = torch.empty(rows, cols, dtype=x.dtype, device=dev)
        dw = db = ws = None
        size = 0
        if params:
            dw, db = torch.empty(cols, dtype=w_dtype, device=dev), torch.empty(cols, dtype=w_dtype, device=dev)
            size = load().fp8_layer_norm_workspace(rows, cols)
            if size < 0:
                _check(size, "fp8_layer_norm_workspace")
            ws = torch.empty(size, dtype=torch.uint8, device=dev)
        st = load().fp8_layer_norm_backward(dy.data_ptr(), _ld(dy), x.data_ptr(), _DTYPES[x.dtype], rows, cols, _ld(x),
                                            _at(weight), _DTYPES[w_dtype], mean.data_ptr(), rstd.data_ptr(),
                                            dx.data_ptr(), cols, _at(dw), _at(db), _at(ws), size, _here(dev))
    _check(st, "fp8_layer_norm_backward")
    return dx, dw, db


class _LayerNormFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, eps):
        y, mean, rstd = layer_norm_forward(x, weight, bias, eps)
        ctx.save_for_backward(x, weight, mean, rstd)
        ctx.has_bias = bias is not None
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        x, weight, mean, rstd = ctx.saved_tensors
        if dy.dtype != x.dtype or dy.stride(-1) != 1 or (dy.shape[0] > 1 and dy.stride(0) < dy.shape[1]):
            dy = _dense(dy.to(x.dtype))
        params = ctx.needs_input_grad[1] or ctx.needs_input_grad[2]
        dx, dw, db = layer_norm_backward(dy, x, weight, mean, rstd, params)
        return (dx if ctx.needs_input_grad[0] else None, dw if ctx.needs_input_grad[1] else None,
                db if ctx.has_bias and ctx.needs_input_grad[2] else None, None)


class LayerNorm(torch.nn.Module):
    """Layer norm over the last dimension, ``features`` long, of BF16 or FP32
    inputs.  ``bias=False`` leaves the shift out.  GPU only, like Linear."""

    def __init__(self, features: int, eps: float = 1e-5, bias: bool = True, device=None, dtype=torch.bfloat16):
        super().__init__()
        if features < 1:
            raise Fp8Error("features must be positive")
        self.features, self.eps = features, eps
        self.weight = torch.nn.Parameter(torch.ones(features, device=device, dtype=dtype))
        self.bias = torch.nn.Parameter(torch.zeros(features, device=device, dtype=dtype)) if bias else None

    def forward(self, x: torch.Tensor) -> torch.Tensor:
        if not x.is_cuda or not self.weight.is_cuda:
            raise Fp8Error("the layer norm runs on the GPU only")
        if x.shape[-1] != self.features:
            raise Fp8Error(f"input has {x.shape[-1]} features, the layer {self.features}")
        if x.dtype not in _DTYPES or self.weight.dtype not in _DTYPES:
            raise Fp8Error("inputs and weights are BF16 or FP32")
        x2d = x.reshape(-1, self.features)
        if x2d.stride(1) != 1 or _ld(x2d) < self.features:
            x2d = _dense(x2d)
        return _LayerNormFn.apply(x2d, self.weight, self.bias, self.eps).reshape(x.shape)


# ---------------------------------------------------------------------------
# RMS norm
# ---------------------------------------------------------------------------

def _like(name: str, t, x) -> None:
    """t is a matrix of x's type and shape (or None)."""
    if t is None:
        return
    if not _is_matrix(t, (x.dtype,)):
        _matrix(name, t, (x.dtype,))
    if t.shape != x.shape:
        raise Fp8Error(f"{name} is {tuple(t.shape)}, x {tuple(x.shape)}")


def rms_norm_forward(x: torch.Tensor, weight: torch.Tensor | None = None, residual: torch.Tensor | None = None,
                     eps: float = 1e-6, stream=None):
    """(y, total, rstd): y the RMS norm of the rows of total = x + residual
    (rounded to x's type; without a residual total is x itself), total and the
    FP32 rstd for rms_norm_backward.  x and residual 2-D with unit column stride."""
    _check_x(x)
    _like("residual", residual, x)
    rows, cols = x.shape
    w_dtype = _params(cols, weight, None)
    _one_device(x, weight, residual)
    dev = x.device
    with _scope(dev, stream):
        y = torch.empty(rows, cols, dtype=x.dtype, device=dev)
        total = x if residual is None else torch.empty(rows, cols, dtype=x.dtype, device=dev)
        rstd = torch.empty(rows, dtype=torch.float32, device=dev)
        st = load().fp8_rms_norm_forward(x.data_ptr(), _DTYPES[x.dtype], rows, cols, _ld(x), _at(residual),
                                         0 if residual is None else _ld(residual), _at(weight), _DTYPES[w_dtype], eps,
                                         None if residual is None else total.data_ptr(), cols, y.data_ptr(), cols,
                                         rstd.data_ptr(), _here(dev))
    _check(st, "fp8_rms_norm_forward")
    return y, total, rstd


def rms_norm_quantize(x: torch.Tensor, recipe: int, fmt: int, orient: int = ROW, weight: torch.Tensor | None = None,
                      residual: torch.Tensor | None = None, eps: float = 1e-6, margin: int = 0,
                      scale: torch.Tensor | None = None, amax: torch.Tensor | None = None,
                      nonfinite: torch.Tensor | None = None, stream=None):
    """(Quantized, total, rstd): rms_norm_forward with the FP8 codes and scales of
    y in its place, cast from the FP32 y.  recipe: BLOCK_1x128, MX_1x32, MX_1x32_OCP,
    or TENSOR_DELAYED with the scale and the amax accumulator of quantize."""
    _check_x(x)
    _like("residual", residual, x)
    if nonfinite is not None:
        _vector("nonfinite", nonfinite, torch.int32, 1)
    rows, cols = x.shape
    w_dtype = _params(cols, weight, None)
    _one_device(x, weight, residual, nonfinite)
    delayed = recipe == TENSOR_DELAYED
    if not delayed and recipe not in (BLOCK_1x128, MX_1x32, MX_1x32_OCP):
        raise Fp8Error("the norm takes the recipes BLOCK_1x128, MX_1x32, MX_1x32_OCP and TENSOR_DELAYED: the others' scales "
                       "need the whole matrix before the first code")
    if not delayed and (scale is not None or amax is not None):
        raise Fp8Error("scale and amax belong to TENSOR_DELAYED")
    dev = x.device
    out = Quantized(fmt=fmt, recipe=recipe, nonfinite=nonfinite)
    ld_r, ld_c = _pad16(cols), _pad16(rows)
    with _scope(dev, stream):
        if orient & ROW:
            out.q_row = torch.empty(rows, ld_r, dtype=torch.uint8, device=dev)
            shp, dt = scale_grid_shape(recipe, rows, cols, ROW)
            if not delayed:
                out.s_row = torch.empty(shp, dtype=dt, device=dev)
        if orient & COL:
            out.q_col = torch.empty(cols, ld_c, dtype=torch.uint8, device=dev)
            shp, dt = scale_grid_shape(recipe, rows, cols, COL)
            if not delayed:
                out.s_col = torch.empty(shp, dtype=dt, device=dev)
        if delayed:
            out.scale = torch.ones(1, dtype=torch.float32, device=dev) if scale is None else scale
            out.amax = torch.zeros(AMAX_SLOTS, dtype=torch.float32, device=dev) if amax is None else amax
            _vector("scale", out.scale, torch.float32, 1)
            _vector("amax", out.amax, torch.float32, AMAX_SLOTS)
            _one_device(x, out.scale, out.amax)
        total = x if residual is None else torch.empty(rows, cols, dtype=x.dtype, device=dev)
        rstd = torch.empty(rows, dtype=torch.float32, device=dev)
        st = load().fp8_rms_norm_quantize(x.data_ptr(), _DTYPES[x.dtype], rows, cols, _ld(x), _at(residual),
                                          0 if residual is None else _ld(residual), _at(weight), _DTYPES[w_dtype], eps,
                                          None if residual is None else total.data_ptr(), cols, rstd.data_ptr(), recipe, fmt,
                                          orient, margin, _at(out.q_row), ld_r, _at(out.s_row), _at(out.q_col), ld_c,
                                          _at(out.s_col), _at(out.scale), _at(out.amax), _at(nonfinite), _here(dev))
    _check(st, "fp8_rms_norm_quantize")
    return out, total, rstd


def rms_norm_backward(dy: torch.Tensor, total: torch.Tensor, weight: torch.Tensor | None, rstd: torch.Tensor,
                      dtotal: torch.Tensor | None = None, params: bool = True, stream=None):
    """(dx, dweight): dx, with dtotal added (the gradient that reaches total by
    itself), is the residual's gradient too; params=False leaves dweight out
    (None).  It takes the weight's dtype, FP32 where there is no weight."""
    _check_x(total)
    if not _is_matrix(dy, (total.dtype,)):
        _matrix("dy", dy, (total.dtype,))
    if dy.shape != total.shape:
        raise Fp8Error(f"dy is {tuple(dy.shape)}, total {tuple(total.shape)}")
    _like("dtotal", dtotal, total)
    rows, cols = total.shape
    w_dtype = _params(cols, weight, None)
    if not _is_vector(rstd, torch.float32, rows):
        _vector("rstd", rstd, torch.float32, rows)
    _one_device(total, dy, weight, rstd, dtotal)
    dev = total.device
    with _scope(dev, stream):
        dx = torch.empty(rows, cols, dtype=total.dtype, device=dev)
        dw = ws = None
        size = 0
        if params:
            dw = torch.empty(cols, dtype=w_dtype, device=dev)
            size = load().fp8_rms_norm_workspace(rows, cols)
            if size < 0:
                _check(size, "fp8_rms_norm_workspace")
            ws = torch.empty(size, dtype=torch.uint8, device=dev)
        st = load().fp8_rms_norm_backward(dy.data_ptr(), _ld(dy), total.data_ptr(), _DTYPES[total.dtype], rows, cols,
                                          _ld(total), _at(weight), _DTYPES[w_dtype], rstd.data_ptr(), _at(dtotal),
                                          0 if dtotal is None else _ld(dtotal), dx.data_ptr(), cols, _at(dw), _at(ws), size,
                                          _here(dev))
    _check(st, "fp8_rms_norm_backward")
    return dx, dw


def _rows_of(t: torch.Tensor, features: int) -> torch.Tensor:
    """t as a matrix of rows that a call takes."""
    t = t.reshape(-1, features)
    return t if t.stride(1) == 1 and _ld(t) >= features else _dense(t)


def _grad_of(d, like: torch.Tensor):
    """A gradient as the kernels take it (None stays None)."""
    if d is None:
        return None
    if d.dtype != like.dtype or d.stride(-1) != 1 or (d.shape[0] > 1 and d.stride(0) < d.shape[1]):
        return _dense(d.to(like.dtype))
    return d


def _rms_norm_grads(dy, total, weight, rstd, dtotal, need_dx: bool, need_dw: bool):
    """dx and dweight where y or total may have no gradient.  dx is always a tensor of its own."""
    if dy is None:
        dw = torch.zeros_like(weight) if need_dw and weight is not None else None
        return dtotal.clone() if need_dx and dtotal is not None else None, dw
    dx, dw = rms_norm_backward(_grad_of(dy, total), total, weight, rstd, _grad_of(dtotal, total), need_dw)
    return dx if need_dx else None, dw


def _read_only(t: torch.Tensor) -> bool:
    """t's gradient goes, through views at most, to a backward pass of this
    package: these read it and hand on tensors of their own."""
    if t.grad_fn is None:
        return False
    made_by = getattr(type((t._base if t._is_view() else t).grad_fn), "_forward_cls", None)
    return made_by is not None and made_by.__module__.rpartition(".")[0] == __package__


def _apart(x: torch.Tensor, residual: torch.Tensor | None) -> bool:
    """The two need gradients in memory of their own.  Autograd takes a gradient
    over as a leaf's .grad, which later passes, hooks and users write to, where it
    sees no other holder of the tensor; behind a view it does not see the other's.
    Where both end in backward passes of this package, neither is written to."""
    return residual is not None and x.requires_grad and residual.requires_grad and not (_read_only(x) and _read_only(residual))


def _to_both(dx, need_x: bool, need_residual: bool, apart: bool):
    """dx as the gradient of x and of the residual."""
    return dx if need_x else None, (dx.clone() if apart and dx is not None else dx) if need_residual else None


class _RMSNormFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, residual, eps):
        ctx.set_materialize_grads(False)
        ctx.apart = _apart(x, residual)
        y, total, rstd = rms_norm_forward(x, weight, residual, eps)
        ctx.save_for_backward(total, weight, rstd)
        return y if residual is None else (y, total)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, dtotal=None):
        total, weight, rstd = ctx.saved_tensors
        need = ctx.needs_input_grad
        dx, dw = _rms_norm_grads(dy, total, weight, rstd, dtotal, need[0] or need[2], need[1])
        dx, dres = _to_both(dx, need[0], need[2], ctx.apart)
        return dx, dw, dres, None


class RMSNorm(torch.nn.Module):
    """RMS norm over the last dimension, ``features`` long, of BF16 or FP32
    inputs.  ``forward(x)`` is the norm; ``forward(x, residual)`` gives (norm of x +
    residual, x + residual), the second for the residual stream.  GPU only, like
    Linear."""

    def __init__(self, features: int, eps: float = 1e-6, device=None, dtype=torch.bfloat16):
        super().__init__()
        if features < 1:
            raise Fp8Error("features must be positive")
        self.features, self.eps = features, eps
        self.weight = torch.nn.Parameter(torch.ones(features, device=device, dtype=dtype))

    def forward(self, x: torch.Tensor, residual: torch.Tensor | None = None):
        _check_layer_input(x, residual, self.weight, self.features)
        x2d = _rows_of(x, self.features)
        if residual is None:
            return _RMSNormFn.apply(x2d, self.weight, None, self.eps).reshape(x.shape)
        y, total = _RMSNormFn.apply(x2d, self.weight, _rows_of(residual, self.features), self.eps)
        return y.reshape(x.shape), total.reshape(x.shape)


def _check_layer_input(x, residual, weight, features: int) -> None:
    if not x.is_cuda or not weight.is_cuda:
        raise Fp8Error("the RMS norm runs on the GPU only")
    if x.shape[-1] != features:
        raise Fp8Error(f"input has {x.shape[-1]} features, the layer {features}")
    if x.dtype not in _DTYPES or weight.dtype not in _DTYPES:
        raise Fp8Error("inputs and weights are BF16 or FP32")
    if residual is not None and (residual.shape != x.shape or residual.dtype != x.dtype or residual.device != x.device):
        raise Fp8Error("x and residual must have one shape, dtype and device")
