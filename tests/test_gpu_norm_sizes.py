"""The layer norm's column sums of more columns than one launch holds (2^32
work-items).

The values are small whole numbers, so that every product and sum below is
exact in binary32 whatever its order, and the results are compared bit for bit."""
import pytest
import torch

import fp8_scaled_quantization_scale_amd as fm
from gpu_util import need_gpu

pytestmark = pytest.mark.gpu

F = torch.float32


def _numbers(n, most):
    """-most .. most, again and again"""
    return (torch.arange(n, dtype=torch.int32, device="cuda") % (2 * most + 1) - most).float()


def _norm_backward(rows, cols, x, dy):
    mean, rstd = torch.zeros(rows, device="cuda"), torch.ones(rows, device="cuda")
    dx = torch.empty(rows, cols, dtype=F, device="cuda")
    out = torch.full((2, cols + 1), 7.0, device="cuda")
    size = fm.fp8_layer_norm_workspace(rows, cols)
    ws = torch.empty(size // 4, device="cuda")
    st = fm.fp8_layer_norm_backward(dy, cols, x, fm.IN_FP32, rows, cols, cols, None, fm.IN_FP32, mean, rstd, dx, cols,
                                    out[0], out[1], ws, size)
    assert st == fm.OK
    assert (out[:, -1] == 7).all()
    return out[0, :-1], out[1, :-1]


def test_column_sums_of_more_columns_than_one_grid_holds():
    """The column sums' second launch takes 64 work-items a column: 2^26 columns."""
    need_gpu()
    cols = (1 << 26) + 35
    x = torch.stack([_numbers(cols, 9), _numbers(cols + 3, 5)[3:]])
    dy = torch.stack([_numbers(cols + 1, 4)[1:], _numbers(cols + 2, 7)[2:]])
    dw, db = _norm_backward(2, cols, x, dy)
    assert torch.equal(dw, (dy * x).sum(0)) and torch.equal(db, dy.sum(0))


@pytest.mark.parametrize("cols", [1 << 26, 1 << 28])
def test_no_rows_of_the_most_columns(cols):
    need_gpu()
    none = torch.empty(0, cols, device="cuda")
    dw, db = _norm_backward(0, cols, none, none)
    assert not dw.any() and not db.any()
