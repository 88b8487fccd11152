"""Layer norm over the libfp8mi C ABI: the layer before an FP8 linear layer.

``layer_norm_forward`` / ``layer_norm_backward`` allocate their outputs with
torch and call the entry points of include/fp8mi.h; ``LayerNorm`` drives them
through autograd.  BF16 or FP32 activations, BF16 or FP32 parameters, FP32
statistics and sums.
"""
from __future__ import annotations

import torch
from torch.autograd.function import once_differentiable

from . import (IN_BF16, IN_FP32, Fp8Error, _at, _check, _dense, _here, _is_matrix, _is_vector, _ld, _matrix, _one_device,
               _scope, _vector, load)

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
