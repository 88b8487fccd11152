"""Inputs of more than 256 MB together are read and written past the caches, by
kernels of their own: each width, type and output against the same rows in pieces
that stay below that.

A row's outputs depend on the row alone, so they are equal bit for bit (transposed
codes and their scales too, in pieces of whole 128-row tiles).  The weight's
gradient adds up r rows in another order: within r + 8 half steps of binary32 of the
sum of magnitudes, from the sum in 64 bits."""
import pytest
import torch

import fp8_scaled_quantization_scale_amd as fm
from fp8_scaled_quantization_scale_amd import norm
from gpu_util import acc_amax, need_gpu

pytestmark = pytest.mark.gpu

E32 = 2.0 ** -24
B, F = torch.bfloat16, torch.float32
WIDTHS = [100, 128, 256, 500, 512, 1000, 1024, 2048, 4000, 4096, 5120, 8192, 16383, 16384]


def _rows(cols, dt, inputs):
    """Just over 256 MB of `inputs` matrices, not a whole number of 128-row tiles."""
    n = (256 << 20) // (inputs * cols * (2 if dt == B else 4))
    return n // 128 * 128 + 128 + 37


def _inputs(rows, cols, dt):
    g = torch.Generator(device="cuda").manual_seed(cols)
    x, res = (torch.randn(rows, cols, generator=g, device="cuda").to(dt) for _ in range(2))
    return x, res, torch.rand(cols, generator=g, device="cuda") + 0.5


def _pieces(rows):
    at = rows // 3 // 128 * 128
    return slice(0, at), slice(at, 2 * at), slice(2 * at, rows)


@pytest.mark.parametrize("dt", [B, F], ids=["bf16", "fp32"])
@pytest.mark.parametrize("cols", WIDTHS)
def test_forward(cols, dt):
    need_gpu()
    rows = _rows(cols, dt, 2)
    x, res, w = _inputs(rows, cols, dt)
    y, total, rstd = norm.rms_norm_forward(x, w, res)
    for s in _pieces(rows):
        a, b, c = norm.rms_norm_forward(x[s], w, res[s])
        assert torch.equal(y[s], a) and torch.equal(total[s], b) and torch.equal(rstd[s], c)


@pytest.mark.parametrize("dt", [B, F], ids=["bf16", "fp32"])
@pytest.mark.parametrize("cols", WIDTHS)
def test_backward(cols, dt):
    need_gpu()
    rows = _rows(cols, dt, 3)
    x, dy, w = _inputs(rows, cols, dt)
    rstd = torch.rand(rows, device="cuda") + 0.5
    dx, dw = norm.rms_norm_backward(dy, x, w, rstd, x)
    s64, size = torch.zeros(cols, dtype=torch.float64, device="cuda"), torch.zeros(cols, dtype=torch.float64, device="cuda")
    for s in _pieces(rows):
        a, _ = norm.rms_norm_backward(dy[s], x[s], w, rstd[s], x[s])
        assert torch.equal(dx[s], a)
        for i in range(s.start, s.stop, max(1, (1 << 24) // cols)):
            at = slice(i, min(s.stop, i + max(1, (1 << 24) // cols)))
            t = dy[at].double() * (x[at].double() * rstd[at, None].double())
            s64, size = s64 + t.sum(0), size + t.abs().sum(0)
    assert ((dw.double() - s64).abs() <= (rows + 8) * E32 * size).all()


RECIPES = [fm.BLOCK_1x128, fm.MX_1x32, fm.MX_1x32_OCP, fm.TENSOR_DELAYED]


@pytest.mark.parametrize("recipe", RECIPES, ids=["block", "mx", "mx_ocp", "delayed"])
@pytest.mark.parametrize("dt", [B, F], ids=["bf16", "fp32"])
@pytest.mark.parametrize("cols", WIDTHS)
def test_codes(cols, dt, recipe):
    need_gpu()
    delayed = recipe == fm.TENSOR_DELAYED
    rows = _rows(cols, dt, 2)
    x, res, w = _inputs(rows, cols, dt)
    fmt = (fm.E4M3, fm.E5M2)[cols % 2]
    for orient in (fm.ROW, fm.ROW_AND_COL, fm.COL):
        if orient == fm.COL and cols not in (100, 4096, 16384):
            continue

        def cast(s):
            more = dict(scale=torch.full((1,), 100.0, device="cuda"), amax=torch.zeros(fm.AMAX_SLOTS, device="cuda")) if delayed else {}
            return norm.rms_norm_quantize(x[s], recipe, fmt, orient, w, res[s], **more)

        q, total, rstd = cast(slice(0, rows))
        most = []
        for s in _pieces(rows):
            p, b, c = cast(s)
            n = b.shape[0]
            assert torch.equal(total[s], b) and torch.equal(rstd[s], c)
            if orient & fm.ROW:
                assert torch.equal(q.q_row[s, :cols], p.q_row[:, :cols]) and (delayed or torch.equal(q.s_row[s], p.s_row))
            if orient & fm.COL:
                assert torch.equal(q.q_col[:, s.start:s.stop], p.q_col[:, :n])
                if not delayed:
                    per = 128 if recipe == fm.BLOCK_1x128 else 32
                    assert torch.equal(q.s_col[:, s.start // per:-(-s.stop // per)], p.s_col)
            if delayed:
                most.append(acc_amax(p.amax))
        assert not delayed or acc_amax(q.amax) == max(most) > 0
