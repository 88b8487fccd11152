"""Layer norm (norm.py) against the formula in float64.

Tolerances, derived before the first run.  A result computed in binary32 and
rounded once to a type with half step u (bf16 2^-8, fp32 2^-24 relative) is off
by at most u |ref| plus the binary32 error of the computation, counted in 2^-24
of the sum of the magnitudes that enter it: the mean and the variance of a row
are sums in trees at most 40 additions deep (8 elements of up to 4 chunks, 6
steps over a wave, 16 waves), and fewer than 60 further operations follow, so
128 steps of 2^-24 cover a row's result (longer rows add one per 8192 columns).
A sum over r rows in any order is off by at most r + 8 steps of the sum of
magnitudes."""
import pytest
import torch

import fp8_scaled_quantization_scale_amd as fm
from fp8_scaled_quantization_scale_amd import norm
from gpu_util import need_gpu

pytestmark = pytest.mark.gpu

E32 = 2.0 ** -24
U = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
B, F = torch.bfloat16, torch.float32

# rows, cols, leading dimension, x dtype, parameter dtype: every register
# variant's border, odd sizes and strides, the rows too long for registers
SHAPES = [
    (1, 1, 1, B, B), (3, 5, 5, F, F), (7, 8, 9, B, F), (64, 511, 511, B, B), (65, 512, 512, B, F), (33, 513, 520, F, B),
    (40, 1000, 1013, B, B), (17, 1024, 1024, F, F), (9, 1025, 1025, B, F), (12, 2048, 2048, B, B), (5, 2049, 2061, F, F),
    (300, 4096, 4096, B, F), (21, 4097, 4097, B, B), (130, 4000, 4200, F, F), (19, 8192, 8192, B, B), (6, 8200, 8200, F, B),
    (600, 16384, 16384, B, B), (11, 16383, 16391, F, F), (5, 16385, 16385, B, B), (7, 40000, 40001, F, B), (2500, 96, 96, B, B),
]


def _inputs(rows, cols, ld, dt, wdt, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed + 31 * rows + cols)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    x = (r(rows, ld) * torch.exp(0.5 * r(1, ld)) + 2.0 * r(rows, 1)).to(dt)[:, :cols]
    return x, (1 + 0.2 * r(cols)).to(wdt), (0.2 * r(cols)).to(wdt), (0.1 * r(rows, ld)).to(dt)[:, :cols]


def _within(got, ref, err, what):
    bad = (got.double() - ref).abs() > U[got.dtype] * ref.abs() + err
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} out of tolerance"


def _reference(x, w, b, eps):
    xd = x.double()
    mean = xd.mean(1, keepdim=True)
    rstd = ((xd - mean).square().mean(1, keepdim=True) + eps).rsqrt()
    h = (xd - mean) * rstd
    wd = 1.0 if w is None else w.double()
    bd = 0.0 if b is None else b.double()
    return mean, rstd, h, wd, bd


def _steps(cols):
    return (128 + cols / 8192) * E32


@pytest.mark.parametrize("rows,cols,ld,dt,wdt", SHAPES)
def test_forward(rows, cols, ld, dt, wdt):
    need_gpu()
    x, w, b, _ = _inputs(rows, cols, ld, dt, wdt)
    for w_, b_ in ((w, b), (w, None), (None, None)) if rows < 50 else ((w, b),):
        y, mean, rstd = norm.layer_norm_forward(x, w_, b_, 1e-5)
        m, r, h, wd, bd = _reference(x, w_, b_, 1e-5)
        size = x.double().abs().mean(1, keepdim=True)
        _within(mean, m[:, 0], (_steps(cols) * size)[:, 0], "mean")
        # the variance moves by the mean's error squared and by its own sum's
        _within(rstd, r[:, 0], (r * _steps(cols))[:, 0], "rstd")
        _within(y, h * wd + bd, _steps(cols) * ((h.abs() + r * size) * abs(wd) + abs(bd)), "y")


@pytest.mark.parametrize("rows,cols,ld,dt,wdt", SHAPES)
def test_backward(rows, cols, ld, dt, wdt):
    need_gpu()
    x, w, _, dy = _inputs(rows, cols, ld, dt, wdt)
    for w_ in (w, None) if rows < 50 else (w,):
        m, r, _, wd, _ = _reference(x, w_, None, 1e-5)
        mean, rstd = m[:, 0].float(), r[:, 0].float()
        dx, dw, db = norm.layer_norm_backward(dy, x, w_, mean, rstd)
        h = (x.double() - mean.double()[:, None]) * rstd.double()[:, None]
        g, rd = dy.double() * wd, rstd.double()[:, None]
        ref = rd * (g - g.mean(1, keepdim=True) - h * (g * h).mean(1, keepdim=True))
        size = rd * (g.abs() + g.abs().mean(1, keepdim=True) + h.abs() * (g * h).abs().mean(1, keepdim=True))
        # h itself is off by two steps of |x - mean| rstd, which cancels against a large mean
        hsize = rd * (x.double().abs() + mean.double().abs()[:, None])
        size = size + rd * (hsize * (g * h).abs().mean(1, keepdim=True) + h.abs() * (g.abs() * hsize).mean(1, keepdim=True))
        _within(dx, ref, _steps(cols) * size, "dx")
        t = dy.double() * h
        _within(dw, t.sum(0), (rows + 8) * E32 * (t.abs() + 2 * dy.double().abs() * hsize).sum(0), "dweight")
        _within(db, dy.double().sum(0), (rows + 8) * E32 * dy.double().abs().sum(0), "dbias")
        assert dw.dtype == db.dtype == (torch.float32 if w_ is None else wdt)
        again = norm.layer_norm_backward(dy, x, w_, mean, rstd)
        assert all(torch.equal(p, q) for p, q in zip((dx, dw, db), again))  # fixed order of addition
        assert norm.layer_norm_backward(dy, x, w_, mean, rstd, params=False)[1:] == (None, None)


def test_neighbours_are_left_alone():
    """Only the columns and rows of the outputs are written (through the C ABI,
    outputs inside larger buffers)."""
    need_gpu()
    rows, cols, ld = 37, 1003, 1050
    x, w, b, dy = _inputs(rows, cols, ld, B, F)
    buf = torch.full((rows + 2, ld), 7.0, dtype=B, device="cuda")
    stats = torch.full((2, rows + 2), 7.0, device="cuda")
    assert fm.fp8_layer_norm_forward(x, fm.IN_BF16, rows, cols, ld, w, b, fm.IN_FP32, 1e-5, buf[1:], ld, stats[0, 1:],
                                     stats[1, 1:]) == fm.OK
    y, mean, rstd = norm.layer_norm_forward(x, w, b)
    assert torch.equal(buf[1:-1, :cols], y) and torch.equal(stats[0, 1:-1], mean) and torch.equal(stats[1, 1:-1], rstd)
    assert (buf[1:-1, cols:] == 7).all() and (buf[0] == 7).all() and (buf[-1] == 7).all()
    assert (stats[:, 0] == 7).all() and (stats[:, -1] == 7).all()
    size = fm.fp8_layer_norm_workspace(rows, cols)
    ws = torch.full((size // 4 + 1,), 7.0, device="cuda")
    out = torch.full((2, cols + 2), 7.0, device="cuda")
    buf.fill_(7.0)
    assert fm.fp8_layer_norm_backward(dy, ld, x, fm.IN_BF16, rows, cols, ld, w, fm.IN_FP32, mean, rstd, buf[1:], ld,
                                      out[0, 1:], out[1, 1:], ws, size) == fm.OK
    dx, dw, db = norm.layer_norm_backward(dy, x, w, mean, rstd)
    assert torch.equal(buf[1:-1, :cols], dx) and torch.equal(out[0, 1:-1], dw) and torch.equal(out[1, 1:-1], db)
    assert (buf[1:-1, cols:] == 7).all() and (buf[0] == 7).all() and (buf[-1] == 7).all() and ws[-1] == 7
    assert (out[:, 0] == 7).all() and (out[:, -1] == 7).all()


def test_no_rows_and_constant_rows():
    need_gpu()
    x = torch.zeros(0, 64, dtype=B, device="cuda")
    w = torch.ones(64, device="cuda")
    y, mean, rstd = norm.layer_norm_forward(x, w, None)
    assert y.shape == (0, 64) and mean.shape == rstd.shape == (0,)
    dx, dw, db = norm.layer_norm_backward(x, x, w, mean, rstd)
    assert dx.shape == (0, 64) and not dw.any() and not db.any()
    # a constant row has variance 0: h is 0 and y the bias, whatever the size of the constant
    x = torch.full((3, 4096), 1e4, dtype=B, device="cuda")
    b = torch.randn(4096, device="cuda")
    y, mean, rstd = norm.layer_norm_forward(x, None, b)
    assert torch.equal(y, b.bfloat16().expand(3, -1)) and torch.allclose(rstd, torch.full_like(rstd, 1e-5 ** -0.5))


def test_nonfinite_stays_in_its_row():
    need_gpu()
    x, w, b, dy = _inputs(9, 700, 700, F, F)
    want, *_ = norm.layer_norm_forward(x, w, b)
    x = x.clone()
    x[2, 5], x[4, 699], x[6, 0] = float("nan"), float("inf"), float("-inf")
    y, mean, rstd = norm.layer_norm_forward(x, w, b)
    hit = torch.tensor([2, 4, 6], device="cuda")
    assert y[hit].isnan().all()
    keep = torch.tensor([0, 1, 3, 5, 7, 8], device="cuda")
    assert torch.equal(y[keep], want[keep])
    dx, _, _ = norm.layer_norm_backward(dy, x, w, mean, rstd)
    assert dx[hit].isnan().all() and dx[keep].isfinite().all()


@pytest.mark.parametrize("dt", [B, F])
def test_layer_gradients(dt):
    """The module against float64 autograd, leading dimensions and a strided input."""
    need_gpu()
    layer = norm.LayerNorm(640, device="cuda", dtype=F)
    with torch.no_grad():
        layer.weight.normal_(1.0, 0.2)
        layer.bias.normal_(0.0, 0.2)
    base = torch.randn(3, 50, 700, device="cuda").to(dt)
    x = base[..., :640].detach().requires_grad_()
    dy = torch.randn(3, 50, 640, device="cuda").to(dt)
    layer(x).backward(dy)
    xr = x.detach().double().requires_grad_()
    wr, br = layer.weight.detach().double().requires_grad_(), layer.bias.detach().double().requires_grad_()
    mu = xr.mean(-1, keepdim=True)
    y = (xr - mu) * ((xr - mu).square().mean(-1, keepdim=True) + layer.eps).rsqrt() * wr + br
    y.backward(dy.double())
    # gradients of size 1: half a step of the type and 1000 binary32 steps
    for got, ref in ((x.grad, xr.grad), (layer.weight.grad, wr.grad), (layer.bias.grad, br.grad)):
        assert ((got.double() - ref).abs() <= U[got.dtype] * ref.abs() + 1000 * E32 * (1 + ref.abs().max())).all()


def test_gradient_against_differences():
    need_gpu()
    x, w, b, dy = _inputs(4, 33, 33, F, F)
    _, mean, rstd = norm.layer_norm_forward(x, w, b, 1e-3)
    dx, dw, db = norm.layer_norm_backward(dy, x, w, mean, rstd)

    def loss(x, w, b):
        m, r, h, wd, bd = _reference(x, w, b, 1e-3)
        return ((h * wd + bd) * dy.double()).sum()

    g = torch.Generator(device="cuda").manual_seed(5)
    for t, grad, at in ((x, dx, 0), (w, dw, 1), (b, db, 2)):
        d = torch.randn(t.shape, generator=g, device="cuda", dtype=torch.float64)
        args = [x.double(), w.double(), b.double()]
        up, down = list(args), list(args)
        up[at], down[at] = args[at] + 1e-5 * d, args[at] - 1e-5 * d
        slope = (loss(*up) - loss(*down)) / 2e-5
        assert abs(slope - (grad.double() * d).sum()) <= 1e-5 * (grad.double() * d).abs().sum() + 1e-8


def test_offsets_past_32_bits():
    """x, y, dy and dx of more than 4 GiB each; the last rows and the sums over all."""
    need_gpu()
    rows, cols = 540000, 4096
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(rows, cols, generator=g, device="cuda", dtype=B)
    w, b = torch.rand(cols, generator=g, device="cuda") + 0.5, torch.rand(cols, generator=g, device="cuda")
    y, mean, rstd = norm.layer_norm_forward(x, w, b)
    few, m, r = norm.layer_norm_forward(x[-3:].clone(), w, b)
    assert torch.equal(y[-3:], few) and torch.equal(mean[-3:], m) and torch.equal(rstd[-3:], r)
    dy = y
    dx, dw, db = norm.layer_norm_backward(dy, x, w, mean, rstd)
    few, _, _ = norm.layer_norm_backward(dy[-3:].clone(), x[-3:].clone(), w, m, r)
    assert torch.equal(dx[-3:], few)
    sdb, adb, sdw, adw = (torch.zeros(cols, dtype=torch.float64, device="cuda") for _ in range(4))
    for i in range(0, rows, 60000):
        d = dy[i:i + 60000].double()
        t = d * (x[i:i + 60000].double() - mean[i:i + 60000, None].double()) * rstd[i:i + 60000, None].double()
        sdb, adb, sdw, adw = sdb + d.sum(0), adb + d.abs().sum(0), sdw + t.sum(0), adw + t.abs().sum(0)
    _within(db, sdb, (rows + 8) * E32 * adb, "dbias")
    _within(dw, sdw, (rows + 8) * E32 * 3 * adw, "dweight")


def test_refusals():
    need_gpu()
    x, w, b, dy = _inputs(8, 64, 64, B, F)
    y, mean, rstd = norm.layer_norm_forward(x, w, b)
    for bad in (lambda: norm.layer_norm_forward(x.half(), w, b), lambda: norm.layer_norm_forward(x[0], w, b),
                lambda: norm.layer_norm_forward(x.t(), w, b), lambda: norm.layer_norm_forward(x, w[:63], b),
                lambda: norm.layer_norm_forward(x, w, b.bfloat16()), lambda: norm.layer_norm_forward(x, w.cpu(), b),
                lambda: norm.layer_norm_forward(x, w, b, -1.0), lambda: norm.layer_norm_forward(x, w, b, float("nan")),
                lambda: norm.layer_norm_forward(x[:, :0], None, None),
                lambda: norm.layer_norm_forward(x[:1].expand(8, 64), w, b),
                lambda: norm.layer_norm_backward(dy.float(), x, w, mean, rstd),
                lambda: norm.layer_norm_backward(dy[:7], x, w, mean, rstd),
                lambda: norm.layer_norm_backward(dy, x, w, mean[:7], rstd),
                lambda: norm.layer_norm_backward(dy, x, w, mean.double(), rstd),
                lambda: norm.LayerNorm(0), lambda: norm.LayerNorm(64)(x), lambda: norm.LayerNorm(32, device="cuda")(x)):
        with pytest.raises(fm.Fp8Error):
            bad()
