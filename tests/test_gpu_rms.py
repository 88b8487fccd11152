"""RMS norm (norm.py) and the norm into FP8 codes against the formula in float64.

Tolerances, derived before the first run, in steps of 2^-24 (half a step of
binary32).  A row's sum of squares has positive terms: a tree of at most 40
additions (8 elements of up to 4 chunks, 6 steps over a wave, 16 waves) after one
rounding each is off by at most 41 steps of itself, rstd by half of that and 4
more, y by two more products: 32 steps of |y| (rows too long for registers add one
addition per 8192 columns, half a step of rstd), and half a step of the type.  dx
subtracts: its terms rstd |g| and rstd |n| mean |g n| are each off by at most 128
steps.  A sum over r rows in any order is off by at most r + 8 steps of the sum of
magnitudes.  The codes and scales are those of the FP32 y, whose three factors are
multiplied in one order: they equal the cast of that product bit for bit."""
import pytest
import torch

import fp8_scaled_quantization_scale_amd as fm
from fp8_scaled_quantization_scale_amd import linear, norm
from gpu_util import acc_amax, need_gpu

pytestmark = pytest.mark.gpu

E32 = 2.0 ** -24
U = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
B, F = torch.bfloat16, torch.float32

# rows, cols, leading dimension, x dtype, weight dtype: every register variant's
# border, odd sizes and strides, the rows too long for registers
SHAPES = [
    (1, 1, 1, B, B), (3, 5, 5, F, F), (7, 8, 9, B, F), (64, 511, 511, B, B), (65, 512, 512, B, F), (33, 513, 520, F, B),
    (40, 1000, 1013, B, B), (17, 1024, 1024, F, F), (9, 1025, 1025, B, F), (12, 2048, 2048, B, B), (5, 2049, 2061, F, F),
    (300, 4096, 4096, B, F), (21, 4097, 4097, B, B), (130, 4000, 4200, F, F), (19, 8192, 8192, B, B), (6, 8200, 8200, F, B),
    (600, 16384, 16384, B, B), (11, 16383, 16391, F, F), (5, 16385, 16385, B, B), (7, 40000, 40001, F, B), (2500, 96, 96, B, B),
]
IDS = [f"{r}x{c}" for r, c, *_ in SHAPES]


def _inputs(rows, cols, ld, dt, wdt, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed + 31 * rows + cols)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    x = (r(rows, ld) * torch.exp(0.5 * r(1, ld))).to(dt)[:, :cols]
    res = (2 * r(rows, ld)).to(dt)[:, :cols]
    return x, res, (1 + 0.2 * r(cols)).to(wdt), (0.1 * r(rows, ld)).to(dt)[:, :cols], (0.1 * r(rows, ld)).to(dt)[:, :cols]


def _within(got, ref, err, what):
    bad = (got.double() - ref).abs() > U[got.dtype] * ref.abs() + err
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} out of tolerance"


def _steps(cols):
    return (32 + cols / 8192) * E32


def _reference(total, w, eps):
    t = total.double()
    rstd = (t.square().mean(1, keepdim=True) + eps) ** -0.5
    return t, rstd, 1.0 if w is None else w.double()


def _sum_of(x, res):
    return x if res is None else (x.float() + res.float()).to(x.dtype)


@pytest.mark.parametrize("rows,cols,ld,dt,wdt", SHAPES, ids=IDS)
def test_forward(rows, cols, ld, dt, wdt):
    need_gpu()
    x, res, w, _, _ = _inputs(rows, cols, ld, dt, wdt)
    for w_, res_ in ((w, res), (w, None), (None, res), (None, None)) if rows < 50 else ((w, res),):
        y, total, rstd = norm.rms_norm_forward(x, w_, res_, 1e-6)
        assert torch.equal(total, _sum_of(x, res_)) and (res_ is not None or total is x)
        t, r, wd = _reference(total, w_, 1e-6)
        _within(rstd, r[:, 0], r[:, 0] * _steps(cols), "rstd")
        _within(y, t * r * wd, (t * r * wd).abs() * _steps(cols), "y")


@pytest.mark.parametrize("rows,cols,ld,dt,wdt", SHAPES, ids=IDS)
def test_backward(rows, cols, ld, dt, wdt):
    need_gpu()
    x, _, w, dy, dt_ = _inputs(rows, cols, ld, dt, wdt)
    for w_, more in ((w, dt_), (w, None), (None, dt_)) if rows < 50 else ((w, dt_),):
        t, r, wd = _reference(x, w_, 1e-6)
        rstd = r[:, 0].float()
        r = rstd.double()[:, None]
        dx, dw = norm.rms_norm_backward(dy, x, w_, rstd, more)
        n, g = t * r, dy.double() * wd
        ref = r * (g - n * (g * n).mean(1, keepdim=True))
        size = r * (g.abs() + n.abs() * (g * n).abs().mean(1, keepdim=True))
        if more is not None:
            ref, size = ref + more.double(), size + more.double().abs()
        _within(dx, ref, (128 + cols / 8192) * E32 * size, "dx")
        s = dy.double() * n
        _within(dw, s.sum(0), (rows + 8) * E32 * s.abs().sum(0), "dweight")
        assert dw.dtype == (F if w_ is None else wdt)
        again = norm.rms_norm_backward(dy, x, w_, rstd, more)
        assert torch.equal(dx, again[0]) and torch.equal(dw, again[1])  # fixed order of addition
        only, none = norm.rms_norm_backward(dy, x, w_, rstd, more, params=False)
        assert none is None and torch.equal(only, dx)


@pytest.mark.parametrize("rows,cols,dt", [(4096, 64, B), (4097, 256, B), (9001, 200, F), (16383, 24, B), (20000, 255, F), (4097, 257, B), (1000, 4000, F),
                                          (16, 128, B), (17, 129, F)])
def test_backward_of_many_short_rows(rows, cols, dt):
    """The numbers of weight-gradient sums on both sides of each change, in a workspace of just the size that is asked for."""
    need_gpu()
    ld = (cols + 7) // 8 * 8
    test_backward(rows, cols, ld, dt, F)
    x, _, w, dy, dt_ = _inputs(rows, cols, ld, dt, F)
    rstd = torch.rand(rows, device="cuda") + 0.5
    dx, dw = norm.rms_norm_backward(dy, x, w, rstd, dt_)
    size = fm.fp8_rms_norm_workspace(rows, cols)
    ws = torch.full((size // 4 + 64,), 7.0, device="cuda")
    got, gw = torch.empty_like(dx), torch.empty_like(dw)
    code = fm.IN_BF16 if dt == B else fm.IN_FP32
    assert fm.fp8_rms_norm_backward(dy, dy.stride(0), x, code, rows, cols, x.stride(0), w, fm.IN_FP32, rstd, dt_, dt_.stride(0),
                                    got, got.stride(0), gw, ws, size) == fm.OK
    assert torch.equal(got, dx) and torch.equal(gw, dw) and (ws[size // 4:] == 7).all()


def _product(total, rstd, w):
    """The FP32 y in a matrix whose rows the cast takes (16-byte multiples)."""
    y = total.float() * rstd[:, None] * (1.0 if w is None else w.float())
    buf = torch.zeros(y.shape[0], (y.shape[1] + 3) // 4 * 4, device="cuda")
    buf[:, : y.shape[1]] = y
    return buf[:, : y.shape[1]]


def _same_codes(q, want, rows, cols, orient):
    if orient & fm.ROW:
        assert torch.equal(q.q_row[:, :cols], want.q_row[:, :cols]), "codes"
        assert torch.equal(q.s_row, want.s_row), "scales"
    if orient & fm.COL:
        assert torch.equal(q.q_col[:, :rows], want.q_col[:, :rows]), "transposed codes"
        assert torch.equal(q.s_col, want.s_col), "transposed scales"


QUANT = [s for s in SHAPES if s[1] <= 40000] + [(1, 128, 128, B, B), (127, 130, 141, B, F), (128, 256, 256, F, F), (129, 33, 33, B, B),
                                                (257, 384, 384, B, F), (33, 1600, 1600, B, B)]


@pytest.mark.parametrize("recipe", [fm.BLOCK_1x128, fm.MX_1x32, fm.MX_1x32_OCP])
@pytest.mark.parametrize("rows,cols,ld,dt,wdt", QUANT, ids=[f"{r}x{c}" for r, c, *_ in QUANT])
def test_codes(rows, cols, ld, dt, wdt, recipe):
    """Codes and scales equal the cast of the FP32 product, total and rstd the
    plain norm's."""
    need_gpu()
    x, res, w, _, _ = _inputs(rows, cols, ld, dt, wdt)
    fmt = (fm.E4M3, fm.E5M2)[(rows + cols + recipe) % 2]
    for orient, w_, res_, margin in ((fm.ROW_AND_COL, w, res, 0), (fm.ROW, w, None, 0), (fm.COL, None, res, 3)):
        margin = margin if recipe == fm.BLOCK_1x128 else 0
        q, total, rstd = norm.rms_norm_quantize(x, recipe, fmt, orient, w_, res_, 1e-6, margin)
        y, total2, rstd2 = norm.rms_norm_forward(x, w_, res_, 1e-6)
        assert torch.equal(total, total2) and torch.equal(rstd, rstd2)
        prod = _product(total, rstd, w_)
        assert torch.equal(y, prod.to(dt))
        _same_codes(q, fm.quantize(prod, recipe, fmt, orient, margin), rows, cols, orient)
        assert (q.q_row is None) == (orient == fm.COL) and (q.q_col is None) == (orient == fm.ROW)


@pytest.mark.parametrize("rows,cols,ld,dt,wdt", QUANT, ids=[f"{r}x{c}" for r, c, *_ in QUANT])
def test_codes_of_delayed_scaling(rows, cols, ld, dt, wdt):
    """Under a scale known beforehand (some values beyond the format's largest): the
    cast's codes of the FP32 product, and its largest magnitude beside what the
    accumulator holds, in every orientation."""
    need_gpu()
    x, res, w, _, _ = _inputs(rows, cols, ld, dt, wdt)
    fmt = (fm.E4M3, fm.E5M2)[(rows + cols) % 2]
    scale = torch.tensor([150.0 if fmt == fm.E4M3 else 20000.0], device="cuda")
    for orient, res_ in ((fm.ROW_AND_COL, res), (fm.ROW, None), (fm.COL, res)):
        amax = torch.zeros(fm.AMAX_SLOTS, device="cuda")
        q, total, rstd = norm.rms_norm_quantize(x, fm.TENSOR_DELAYED, fmt, orient, w, res_, scale=scale, amax=amax)
        prod = _product(total, rstd, w)
        want = fm.quantize(prod, fm.TENSOR_DELAYED, fmt, orient, scale=scale)
        if orient & fm.ROW:
            assert torch.equal(q.q_row[:, :cols], want.q_row[:, :cols])
        if orient & fm.COL:
            assert torch.equal(q.q_col[:, :rows], want.q_col[:, :rows])
        assert q.amax is amax and acc_amax(amax) == acc_amax(want.amax) == prod.abs().max().item()
        norm.rms_norm_quantize(0.5 * x, fm.TENSOR_DELAYED, fmt, orient, None, None, scale=scale, amax=amax)
        assert acc_amax(amax) >= acc_amax(want.amax)
    bad = x.clone()
    bad[rows // 2, cols // 2] = float("nan")
    amax = torch.zeros(fm.AMAX_SLOTS, device="cuda")
    q, _, rstd = norm.rms_norm_quantize(bad, fm.TENSOR_DELAYED, fmt, fm.ROW_AND_COL, w, None, scale=scale, amax=amax)
    want = fm.quantize(_product(bad, rstd, w), fm.TENSOR_DELAYED, fmt, fm.ROW_AND_COL, scale=scale)
    assert torch.equal(q.q_row[:, :cols], want.q_row[:, :cols]) and torch.equal(q.q_col[:, :rows], want.q_col[:, :rows])
    assert acc_amax(amax) != acc_amax(amax)


@pytest.mark.parametrize("rows,cols,ld,dt,wdt", [(1, 128, 128, B, F), (17, 129, 136, F, B), (33, 255, 261, B, B), (31, 127, 129, F, F),
                                                 (70001, 128, 128, B, B), (35000, 256, 256, F, F), (40003, 72, 80, B, F)])
def test_rows_of_a_quarter_wave(rows, cols, ld, dt, wdt):
    """Four rows to a wave: each path at the widths where the split changes, and with more rows than are held at once, so that
    the last round leaves some of a wave's rows without work."""
    test_forward(rows, cols, ld, dt, wdt)
    test_backward(rows, cols, ld, dt, wdt)
    for recipe in (fm.BLOCK_1x128, fm.MX_1x32, fm.MX_1x32_OCP):
        test_codes(rows, cols, ld, dt, wdt, recipe)
    test_codes_of_delayed_scaling(rows, cols, ld, dt, wdt)


@pytest.mark.parametrize("fmt,u,least", [(fm.E4M3, 2.0 ** -4, 2.0 ** -10), (fm.E5M2, 2.0 ** -3, 2.0 ** -17)])
def test_codes_stand_for_the_norm(fmt, u, least):
    """Codes times scales against y in 64 bits: half a step of the code's value, or
    of the smallest one, and the scale's and y's own roundings."""
    need_gpu()
    x, res, w, _, _ = _inputs(200, 700, 700, B, F)
    q, total, rstd = norm.rms_norm_quantize(x, fm.BLOCK_1x128, fmt, fm.ROW_AND_COL, w, res)
    t, r, wd = _reference(total, w, 1e-6)
    for codes, scales, ref in ((q.q_row[:, :700], q.s_row, t * r * wd), (q.q_col[:, :200], q.s_col, (t * r * wd).t())):
        s = scales.double().repeat_interleave(128, 1)[:, : codes.shape[1]]
        v = codes.view(fm.TORCH_FP8[fmt]).double() * s
        assert ((v - ref).abs() <= u * ref.abs() + least * s + 40 * E32 * ref.abs()).all()


def test_neighbours_are_left_alone():
    """Only the columns and rows of the outputs are written (through the C ABI,
    outputs inside larger buffers)."""
    need_gpu()
    rows, cols, ld = 37, 1003, 1050
    x, res, w, dy, dt_ = _inputs(rows, cols, ld, B, F)
    y, total, rstd = norm.rms_norm_forward(x, w, res)
    out = torch.full((2, rows + 2, ld), 7.0, dtype=B, device="cuda")
    st = torch.full((rows + 2,), 7.0, device="cuda")
    assert fm.fp8_rms_norm_forward(x, fm.IN_BF16, rows, cols, ld, res, ld, w, fm.IN_FP32, 1e-6, out[0, 1:], ld, out[1, 1:], ld,
                                   st[1:]) == fm.OK
    assert torch.equal(out[0, 1:-1, :cols], total) and torch.equal(out[1, 1:-1, :cols], y) and torch.equal(st[1:-1], rstd)
    assert (out[:, 1:-1, cols:] == 7).all() and (out[:, 0] == 7).all() and (out[:, -1] == 7).all() and st[0] == st[-1] == 7
    for recipe, per, dtype in ((fm.BLOCK_1x128, 128, F), (fm.MX_1x32, 32, torch.uint8)):
        q, _, _ = norm.rms_norm_quantize(x, recipe, fm.E4M3, fm.ROW_AND_COL, w, res)
        cr = torch.full((rows + 2, 1056), 7, dtype=torch.uint8, device="cuda")
        cc = torch.full((cols + 2, 64), 7, dtype=torch.uint8, device="cuda")
        nr, nc = rows * -(-cols // per), cols * -(-rows // per)
        sr, sc = (torch.full((n + 8,), 7, device="cuda").to(dtype) for n in (nr, nc))
        assert fm.fp8_rms_norm_quantize(x, fm.IN_BF16, rows, cols, ld, res, ld, w, fm.IN_FP32, 1e-6, out[0, 1:], ld, st[1:],
                                        recipe, fm.E4M3, fm.ROW_AND_COL, 0, cr[1:], 1056, sr[4:], cc[1:], 64, sc[4:], None, None, None) == fm.OK
        assert torch.equal(cr[1:-1, :cols], q.q_row[:, :cols]) and torch.equal(cc[1:-1, :rows], q.q_col[:, :rows])
        assert (cr[1:-1, cols:] == 7).all() and (cr[0] == 7).all() and (cr[-1] == 7).all()
        assert (cc[1:-1, rows:] == 7).all() and (cc[0] == 7).all() and (cc[-1] == 7).all()
        assert torch.equal(sr[4:4 + nr], q.s_row.reshape(-1)) and (sr[:4] == 7).all() and (sr[4 + nr:] == 7).all()
        assert torch.equal(sc[4:4 + nc], q.s_col.reshape(-1)) and (sc[:4] == 7).all() and (sc[4 + nc:] == 7).all()
    size = fm.fp8_rms_norm_workspace(rows, cols)
    ws = torch.full((size // 4 + 1,), 7.0, device="cuda")
    dw = torch.full((cols + 2,), 7.0, device="cuda")
    out.fill_(7.0)
    assert fm.fp8_rms_norm_backward(dy, ld, x, fm.IN_BF16, rows, cols, ld, w, fm.IN_FP32, rstd, dt_, ld, out[0, 1:], ld, dw[1:], ws,
                                    size) == fm.OK
    dx, want = norm.rms_norm_backward(dy, x, w, rstd, dt_)
    assert torch.equal(out[0, 1:-1, :cols], dx) and torch.equal(dw[1:-1], want) and dw[0] == dw[-1] == ws[-1] == 7
    assert (out[0, 1:-1, cols:] == 7).all() and (out[0, 0] == 7).all() and (out[0, -1] == 7).all()


def test_no_rows_and_rows_of_zeros():
    need_gpu()
    x = torch.zeros(0, 64, dtype=B, device="cuda")
    w = torch.ones(64, device="cuda")
    y, total, rstd = norm.rms_norm_forward(x, w, x)
    assert y.shape == total.shape == (0, 64) and rstd.shape == (0,)
    q, _, _ = norm.rms_norm_quantize(x, fm.BLOCK_1x128, fm.E4M3, fm.ROW_AND_COL, w, x)
    assert q.q_row.shape[0] == 0 and q.s_col.shape == (64, 0)
    dx, dw = norm.rms_norm_backward(x, x, w, rstd, x)
    assert dx.shape == (0, 64) and not dw.any()
    # a row of zeros is zeros; its blocks have scale 1
    x = torch.zeros(3, 4096, dtype=B, device="cuda")
    y, _, rstd = norm.rms_norm_forward(x, None, None, 1e-6)
    assert not y.any() and torch.allclose(rstd, torch.full_like(rstd, 1e3))
    q, _, _ = norm.rms_norm_quantize(x, fm.BLOCK_1x128, fm.E4M3, fm.ROW_AND_COL)
    assert not q.q_row.any() and not q.q_col[:, :3].any() and (q.s_row == 1).all() and (q.s_col == 1).all()


@pytest.mark.parametrize("recipe", [fm.BLOCK_1x128, fm.MX_1x32])
def test_nonfinite_stays_in_its_row(recipe):
    need_gpu()
    x, _, w, dy, _ = _inputs(9, 700, 700, F, F)
    want, *_ = norm.rms_norm_forward(x, w)
    bad = x.clone()
    bad[2, 5], bad[4, 699], bad[6, 0] = float("nan"), float("inf"), float("-inf")
    y, total, rstd = norm.rms_norm_forward(bad, w)
    keep = torch.tensor([0, 1, 3, 5, 7, 8], device="cuda")
    assert torch.equal(y[keep], want[keep]) and y[2].isnan().all() and y[4, 699].isnan() and y[6, 0].isnan()
    dx, _ = norm.rms_norm_backward(dy, bad, w, rstd)
    assert dx[keep].isfinite().all() and dx[2].isnan().all()
    # codes: the cast's own treatment of such blocks, and its count of them
    count, count2 = (torch.zeros(1, dtype=torch.int32, device="cuda") for _ in range(2))
    q, _, _ = norm.rms_norm_quantize(bad, recipe, fm.E4M3, fm.ROW_AND_COL, w, nonfinite=count)
    _same_codes(q, fm.quantize(_product(bad, rstd, w), recipe, fm.E4M3, fm.ROW_AND_COL, nonfinite=count2), 9, 700, fm.ROW_AND_COL)
    assert count.item() == count2.item() > 0


def _plain(x, res, w, eps):
    total = x if res is None else x + res
    return total * (total.square().mean(-1, keepdim=True) + eps) ** -0.5 * w, total


@pytest.mark.parametrize("dt", [B, F])
@pytest.mark.parametrize("residual", [False, True])
def test_layer_gradients(dt, residual):
    """The module against float64 autograd, leading dimensions and strided inputs,
    with a gradient along the residual stream."""
    need_gpu()
    layer = norm.RMSNorm(640, device="cuda", dtype=F)
    with torch.no_grad():
        layer.weight.normal_(1.0, 0.2)
    x = torch.randn(3, 50, 700, device="cuda").to(dt)[..., :640].detach().requires_grad_()
    res = torch.randn(3, 50, 640, device="cuda").to(dt).requires_grad_()
    dy, dtotal = (torch.randn(3, 50, 640, device="cuda").to(dt) for _ in range(2))
    wr = layer.weight.detach().double().requires_grad_()
    if residual:
        y, total = layer(x, res)
        torch.autograd.backward([y, total], [dy, dtotal])
        assert torch.equal(x.grad, res.grad)
        xr = total.detach().double().requires_grad_()
        torch.autograd.backward([_plain(xr, None, wr, layer.eps)[0], xr * 1.0], [dy.double(), dtotal.double()])
    else:
        layer(x).backward(dy)
        xr = x.detach().double().requires_grad_()
        _plain(xr, None, wr, layer.eps)[0].backward(dy.double())
    for got, ref in ((x.grad, xr.grad), (layer.weight.grad, wr.grad)):  # gradients of size 1: 1000 binary32 steps
        assert ((got.double() - ref).abs() <= U[got.dtype] * ref.abs() + 1000 * E32 * (1 + ref.abs().max())).all()


def test_layer_uses_one_output_or_the_other():
    """A gradient of y alone, of total alone, and frozen inputs."""
    need_gpu()
    layer = norm.RMSNorm(256, device="cuda", dtype=F)
    x, res = (torch.randn(20, 256, device="cuda").requires_grad_() for _ in range(2))
    y, total = layer(x, res)
    total.sum().backward()
    assert (x.grad == 1).all() and (res.grad == 1).all() and not layer.weight.grad.any()
    x.grad = res.grad = layer.weight.grad = None
    y, _ = layer(x, res)
    y.sum().backward()
    dx, dw = norm.rms_norm_backward(torch.ones_like(y), (x + res).detach(), layer.weight.detach(),
                                    norm.rms_norm_forward((x + res).detach(), layer.weight.detach())[2])
    assert torch.equal(x.grad, dx) and torch.equal(layer.weight.grad, dw)
    layer.weight.requires_grad_(False)
    x.grad = None
    y, _ = layer(x, res.detach())
    y.sum().backward()
    assert torch.equal(x.grad, dx)
    with torch.no_grad():
        assert torch.equal(layer(x, res)[0], y)


def test_gradient_against_differences():
    need_gpu()
    x, _, w, dy, _ = _inputs(4, 33, 33, F, F)
    _, _, rstd = norm.rms_norm_forward(x, w, None, 1e-3)
    dx, dw = norm.rms_norm_backward(dy, x, w, rstd)

    def loss(x, w):
        return (_plain(x, None, w, 1e-3)[0] * dy.double()).sum()

    g = torch.Generator(device="cuda").manual_seed(5)
    for t, grad, at in ((x, dx, 0), (w, dw, 1)):
        d = torch.randn(t.shape, generator=g, device="cuda", dtype=torch.float64)
        args = [x.double(), w.double()]
        up, down = list(args), list(args)
        up[at], down[at] = args[at] + 1e-5 * d, args[at] - 1e-5 * d
        slope = (loss(*up) - loss(*down)) / 2e-5
        assert abs(slope - (grad.double() * d).sum()) <= 1e-5 * (grad.double() * d).abs().sum() + 1e-8


@pytest.mark.parametrize("recipe", [linear.Float8BlockScaling(), linear.Float8BlockScaling(linear.Format.HYBRID), linear.MXFP8BlockScaling()])
@pytest.mark.parametrize("dt", [B, F])
def test_norm_linear(recipe, dt):
    """RMSNormLinear makes the calls that its parts make one by one: the product of
    the norm's codes, and in the backward pass the products and the norm's."""
    need_gpu()
    layer = linear.RMSNormLinear(384, 320, recipe=recipe, device="cuda", dtype=dt)
    with torch.no_grad():
        layer.norm_weight.normal_(1.0, 0.2)
    x, res, dtotal = (torch.randn(2, 136, 384, device="cuda").to(dt) for _ in range(3))
    dy = (1e-2 * torch.randn(2, 136, 320, device="cuda")).to(dt)
    x.requires_grad_()
    res.requires_grad_()
    y, total = layer(x, res)
    torch.autograd.backward([y, total], [dy, dtotal])
    p = linear.plan(recipe)
    (rx, fx), (rw, fw), (rg, fg) = (p.quant[k] for k in "xwg")
    w, nw = layer.weight.detach(), layer.norm_weight.detach()
    q, t2, rstd = norm.rms_norm_quantize(x.detach().view(272, 384), rx, fx, fm.ROW_AND_COL, nw, res.detach().view(272, 384), layer.eps)
    qw, qg = fm.quantize(w, rw, fw, fm.ROW_AND_COL), fm.quantize(dy.view(272, 320), rg, fg, fm.ROW_AND_COL)
    assert torch.equal(total.view(272, 384), t2)
    assert torch.equal(y.view(272, 320), fm.gemm(q.q_row, fx, q.s_row, qw.q_row, fw, qw.s_row, p.gemm["fprop"], 384, dt))
    dn = fm.gemm(qg.q_row, fg, qg.s_row, qw.q_col, fw, qw.s_col, p.gemm["dgrad"], 320, dt, M=272, N=384)
    dw = fm.gemm(qg.q_col, fg, qg.s_col, q.q_col, fx, q.s_col, p.gemm["wgrad"], 272, dt, M=320, N=384)
    dx, dnw = norm.rms_norm_backward(dn, t2, nw, rstd, dtotal.view(272, 384))
    assert torch.equal(layer.weight.grad, dw) and torch.equal(layer.norm_weight.grad, dnw)
    assert torch.equal(x.grad.view(272, 384), dx) and torch.equal(res.grad, x.grad)
    # near the layers one by one, whose norm is rounded to x's type before the cast
    separate = linear.Linear(384, 320, recipe=recipe, device="cuda", dtype=dt)
    separate.weight.data.copy_(w)
    n, _, _ = norm.rms_norm_forward(t2, nw, None, layer.eps)
    z = separate(n)
    assert (z - y.view(272, 320)).norm() <= 0.03 * z.norm()
    with torch.no_grad():
        assert torch.equal(layer(x, res)[0], y) and torch.equal(layer(total), y)


@pytest.mark.parametrize("interval", [1, 2])
def test_norm_linear_delayed_scaling(interval):
    """The same under delayed scaling, over steps that update the scales; the state
    travels with the module."""
    need_gpu()
    rec = linear.DelayedScaling(interval=interval, amax_history_len=4)
    torch.manual_seed(1)
    layer = linear.RMSNormLinear(256, 128, recipe=rec, device="cuda")
    length, margin, fwd, bwd = 4, 0, fm.E4M3, fm.E5M2
    sx, sw, sg = (fm.DelayedState(f, length, margin) for f in (fwd, fwd, bwd))
    w, nw = layer.weight.detach(), layer.norm_weight.detach()
    for step in range(1, 6):
        x = (step * torch.randn(64, 256, device="cuda")).bfloat16().requires_grad_()
        res, dtotal = (torch.randn(64, 256, device="cuda").bfloat16() for _ in range(2))
        dy = (1e-3 * torch.randn(64, 128, device="cuda")).bfloat16()
        layer.weight.grad = layer.norm_weight.grad = None
        y, total = layer(x, res)
        torch.autograd.backward([y, total], [dy, dtotal])
        q, t2, rstd = norm.rms_norm_quantize(x.detach(), fm.TENSOR_DELAYED, fwd, fm.ROW_AND_COL, nw, res, layer.eps, scale=sx.scale,
                                             amax=sx.amax)
        ix = sx.scale_inv.clone()
        qw, qg = sw.quantize(w, fm.ROW_AND_COL), sg.quantize(dy, fm.ROW_AND_COL)
        assert torch.equal(total, t2) and torch.equal(y, fm.gemm(q.q_row, fwd, ix, qw.q_row, fwd, qw.scale_inv, fm.GEMM_TENSOR, 256))
        dn = fm.gemm(qg.q_row, bwd, qg.scale_inv, qw.q_col, fwd, qw.scale_inv, fm.GEMM_TENSOR, 128, M=64, N=256)
        dw = fm.gemm(qg.q_col, bwd, qg.scale_inv, q.q_col, fwd, ix, fm.GEMM_TENSOR, 64, M=128, N=256)
        dx, dnw = norm.rms_norm_backward(dn, t2, nw, rstd, dtotal)
        assert torch.equal(x.grad, dx) and torch.equal(layer.weight.grad, dw) and torch.equal(layer.norm_weight.grad, dnw)
        if step % interval == 0:
            for s in (sx, sw, sg):
                s.update()
    assert sx.scale.item() != 1.0
    other = linear.RMSNormLinear(256, 128, recipe=rec, device="cuda")
    other.load_state_dict(layer.state_dict())
    with torch.no_grad():
        assert torch.equal(other(x, res)[0], layer(x, res)[0])


def test_norm_linear_grad_of_total_alone_and_frozen_weight():
    need_gpu()
    layer = linear.RMSNormLinear(128, 64, recipe=linear.Float8BlockScaling(), device="cuda")
    x, res = (torch.randn(16, 128, device="cuda").bfloat16().requires_grad_() for _ in range(2))
    _, total = layer(x, res)
    total.float().sum().backward()
    assert (x.grad == 1).all() and not layer.weight.grad.any() and not layer.norm_weight.grad.any()
    x.grad = None
    layer.weight.requires_grad_(False)
    x7 = torch.randn(7, 128, device="cuda").bfloat16().requires_grad_()  # no weight gradient: any number of tokens
    layer(x7).float().sum().backward()
    assert x7.grad.isfinite().all() and x7.grad.any()


def test_side_stream_and_captured_replays():
    """On a stream given, and a training step of norm and product in a graph,
    replayed with other inputs between eager work."""
    need_gpu()
    x, res, w, _, _ = _inputs(256, 512, 512, B, F)
    want = norm.rms_norm_quantize(x, fm.BLOCK_1x128, fm.E4M3, fm.ROW_AND_COL, w, res)
    torch.cuda.synchronize()
    for raw in (False, True):
        s = torch.cuda.Stream()
        got = norm.rms_norm_quantize(x, fm.BLOCK_1x128, fm.E4M3, fm.ROW_AND_COL, w, res, stream=s.cuda_stream if raw else s)
        s.synchronize()
        assert torch.equal(got[0].q_col, want[0].q_col) and torch.equal(got[0].s_row, want[0].s_row) and torch.equal(got[1], want[1])
    layer = linear.RMSNormLinear(512, 256, recipe=linear.Float8BlockScaling(), device="cuda")
    params = (layer.norm_weight, layer.weight)

    def step(x, res, dy):
        x, res = x.detach().requires_grad_(), res.detach().requires_grad_()
        y, total = layer(x, res)
        grads = torch.autograd.grad([y, total], [x, res, *params], [dy, total.detach()])
        return tuple(t.detach() for t in (y, total, *grads))  # (no graph outlives its step)

    def inputs(seed):
        a, b, _, _, _ = _inputs(256, 512, 512, B, F, seed)
        return a, b, _inputs(256, 256, 256, B, F, seed)[3]

    static = [t.clone() for t in inputs(1)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(2):
            step(*static)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(*static)
    for seed in (2, 3, 4, 1):
        fresh = inputs(seed)
        want = step(*fresh)
        torch.cuda.synchronize()
        for a, b in zip(static, fresh):
            a.copy_(b)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want)), seed


def test_offsets_past_32_bits():
    """Rows and codes of more than 4 GiB each; the last rows and the sums over all."""
    need_gpu()
    rows, cols = 1048576 + 200, 4096
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(rows, cols, generator=g, device="cuda", dtype=B)
    w = torch.rand(cols, generator=g, device="cuda") + 0.5
    q, total, rstd = norm.rms_norm_quantize(x, fm.BLOCK_1x128, fm.E4M3, fm.ROW_AND_COL, w, x)
    few = norm.rms_norm_quantize(x[-72:].clone(), fm.BLOCK_1x128, fm.E4M3, fm.ROW_AND_COL, w, x[-72:].clone())  # a last row tile
    assert torch.equal(total[-72:], few[1]) and torch.equal(rstd[-72:], few[2]) and torch.equal(q.q_row[-72:], few[0].q_row)
    assert torch.equal(q.s_row[-72:], few[0].s_row) and torch.equal(q.q_col[:, rows - 72:rows], few[0].q_col[:, :72])
    assert torch.equal(q.s_col[:, -1:], few[0].s_col)
    del q
    y, _, _ = norm.rms_norm_forward(total, w)
    assert torch.equal(y[-72:], norm.rms_norm_forward(total[-72:].clone(), w)[0])
    dx, dw = norm.rms_norm_backward(y, total, w, rstd, x)
    few, _ = norm.rms_norm_backward(y[-3:].clone(), total[-3:].clone(), w, rstd[-3:].clone(), x[-3:].clone())
    assert torch.equal(dx[-3:], few)
    s, a = torch.zeros(cols, dtype=torch.float64, device="cuda"), torch.zeros(cols, dtype=torch.float64, device="cuda")
    for i in range(0, rows, 65536):
        t = y[i:i + 65536].double() * (total[i:i + 65536].double() * rstd[i:i + 65536, None].double())
        s, a = s + t.sum(0), a + t.abs().sum(0)
    _within(dw, s, (rows + 8) * E32 * a, "dweight")


def test_more_columns_than_one_launch_adds():
    """From 2^26 columns on the weight's sums go out as several launches."""
    need_gpu()
    rows, cols = 2, (1 << 26) + 43
    g = torch.Generator(device="cuda").manual_seed(9)
    x, dy = (torch.randn(rows, cols, generator=g, device="cuda", dtype=B) for _ in range(2))
    w = (torch.rand(cols, generator=g, device="cuda") + 0.5).to(B)
    y, _, rstd = norm.rms_norm_forward(x, w)
    assert ((rstd.double() ** -2 - 1e-6) / torch.stack([r.double().square().mean() for r in x]) - 1).abs().max() <= 2 * _steps(cols)
    dx, dw = norm.rms_norm_backward(dy, x, w, rstd)
    r = rstd.double()[:, None]
    mean = sum(((dy[:, i:i + (1 << 24)].double() * w[i:i + (1 << 24)].double()) * (x[:, i:i + (1 << 24)].double() * r)).sum(1, keepdim=True)
               for i in range(0, cols, 1 << 24)) / cols
    for at in (slice(0, 1000), slice((1 << 26) - 500, cols)):
        n, d, wd = x[:, at].double() * r, dy[:, at].double(), w[at].double()
        _within(y[:, at], n * wd, (n * wd).abs() * _steps(cols), "y")
        _within(dw[at], (d * n).sum(0), (rows + 8) * E32 * (d * n).abs().sum(0), "dweight")
        # the mean's own error is a part of its terms' mean size, 1 here, which dominates it
        _within(dx[:, at], r * (d * wd - n * mean), (128 + cols / 8192) * E32 * r * ((d * wd).abs() + n.abs()), "dx")


def test_refusals():
    need_gpu()
    x, res, w, dy, _ = _inputs(8, 64, 64, B, F)
    y, total, rstd = norm.rms_norm_forward(x, w, res)
    fwd, quant, back = norm.rms_norm_forward, norm.rms_norm_quantize, norm.rms_norm_backward
    block = fm.BLOCK_1x128
    rec = linear.Float8BlockScaling()
    layer = linear.RMSNormLinear(64, 64, recipe=rec, device="cuda")
    for bad in (lambda: fwd(x.half(), w), lambda: fwd(x[0], w), lambda: fwd(x.t(), w), lambda: fwd(x, w[:63]), lambda: fwd(x, w.cpu()),
                lambda: fwd(x, w, res.float()), lambda: fwd(x, w, res[:7]), lambda: fwd(x, w, res.cpu()), lambda: fwd(x, w, res, -1.0),
                lambda: fwd(x, w, res, float("nan")), lambda: fwd(x[:, :0]), lambda: fwd(x[:1].expand(8, 64), w),
                lambda: fwd(x, w, res[:1].expand(8, 64)),
                lambda: quant(x, fm.TENSOR_CURRENT, fm.E4M3), lambda: quant(x, fm.BLOCK_128x128, fm.E4M3), lambda: quant(x, fm.CHANNEL, fm.E4M3),
                lambda: quant(x, block, 2), lambda: quant(x, block, fm.E4M3, 0), lambda: quant(x, block, fm.E4M3, 4),
                lambda: quant(x, block, fm.E4M3, margin=65), lambda: quant(x, block, fm.E4M3, eps=-1.0),
                lambda: quant(x, block, fm.E4M3, nonfinite=torch.zeros(1, device="cuda")),
                lambda: back(dy.float(), x, w, rstd), lambda: back(dy[:7], x, w, rstd), lambda: back(dy, x, w, rstd[:7]),
                lambda: back(dy, x, w, rstd.double()), lambda: back(dy, x, w, rstd, dy.float()), lambda: back(dy, x, w, rstd, dy[:, :63]),
                lambda: norm.RMSNorm(0), lambda: norm.RMSNorm(64)(x), lambda: norm.RMSNorm(32, device="cuda")(x),
                lambda: norm.RMSNorm(64, device="cuda")(x, res.float()), lambda: norm.RMSNorm(64, device="cuda")(x, res[:4]),
                lambda: linear.RMSNormLinear(40, 64), lambda: linear.RMSNormLinear(64, 64, device="cuda")(x),
                lambda: linear.RMSNormLinear(64, 64, recipe=linear.Float8CurrentScaling(), device="cuda")(x),
                lambda: linear.RMSNormLinear(64, 64, recipe=linear.Float8ChannelScaling(), device="cuda")(x),
                lambda: quant(x, block, fm.E4M3, scale=rstd), lambda: quant(x, fm.TENSOR_DELAYED, fm.E4M3, amax=rstd),
                lambda: quant(x, fm.TENSOR_DELAYED, fm.E4M3, scale=rstd.double()),
                lambda: layer(x), lambda: layer(x[:, :32]), lambda: layer(x, res[:4])):
        with pytest.raises(fm.Fp8Error):
            bad()


def test_no_second_derivative():
    need_gpu()
    x = torch.randn(16, 128, device="cuda", requires_grad=True)
    for f in (norm.RMSNorm(128, device="cuda", dtype=F), linear.RMSNormLinear(128, 64, recipe=linear.Float8BlockScaling(), device="cuda", dtype=F)):
        g, = torch.autograd.grad(f(x).square().sum(), x, create_graph=True)
        with pytest.raises(RuntimeError):
            g.sum().backward()
