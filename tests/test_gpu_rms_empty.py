"""RMSNorm, RMSNormLinear, the router and its balance on no tokens, with empty
tensors of any strides, and the norm with eps = 0."""
import pytest
import torch

import fp8_scaled_quantization_scale_amd as fm
from fp8_scaled_quantization_scale_amd import linear, moe, norm
from gpu_util import need_gpu

pytestmark = pytest.mark.gpu

RECIPES = [linear.Float8BlockScaling(), linear.MXFP8BlockScaling(), linear.DelayedScaling()]
B, F = torch.bfloat16, torch.float32

EMPTY = {
    "row-major": lambda dt: torch.empty(0, 256, dtype=dt, device="cuda"),
    "expanded": lambda dt: torch.zeros((), dtype=dt, device="cuda").expand(0, 256),
    "transposed": lambda dt: torch.empty(256, 0, dtype=dt, device="cuda").t(),
    "every other": lambda dt: torch.empty(0, 512, dtype=dt, device="cuda")[:, ::2],
    "three dimensions": lambda dt: torch.empty(4, 0, 256, dtype=dt, device="cuda"),
    "a slice": lambda dt: torch.empty(5, 300, dtype=dt, device="cuda")[2:2, :256],
}


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("how", EMPTY)
@pytest.mark.parametrize("which", ["norm"] + RECIPES, ids=["norm", "block", "mx", "delayed"])
def test_layers(which, how, residual):
    need_gpu()
    for dt in (B, F):
        layer = (norm.RMSNorm(256, device="cuda", dtype=dt) if which == "norm" else
                 linear.RMSNormLinear(256, 128, recipe=which, device="cuda", dtype=dt))
        x, res = (EMPTY[how](dt).detach().requires_grad_() for _ in range(2))
        out = layer(x, res) if residual else (layer(x),)
        assert out[0].shape == (*x.shape[:-1], 256 if which == "norm" else 128) and out[0].dtype == dt
        if residual:
            assert out[1].shape == x.shape and out[1].dtype == dt
        sum(t.sum() for t in out).backward()
        assert x.grad.shape == x.shape and (not residual or res.grad.shape == res.shape)
        for p in layer.parameters():
            assert p.grad.shape == p.shape and not p.grad.any()
        if residual:  # total alone
            layer(x, res)[1].sum().backward()
        with torch.no_grad():
            layer(x, res) if residual else layer(x)


@pytest.mark.parametrize("dt", [B, F])
def test_router(dt):
    need_gpu()
    for l in (torch.empty(0, 8, dtype=dt, device="cuda"), torch.empty(0, 20, dtype=dt, device="cuda")[:, :8]):
        l = l.detach().requires_grad_()
        for mask in (None, torch.empty(0, dtype=torch.bool, device="cuda")):
            r = moe.route(l, 2, mask=mask)
            assert r.expert.shape == r.weights.shape == (0, 2) and r.loss == 0 and not r.counts.any() and not r.slope.any()
            g, = torch.autograd.grad(r.weights.sum() + r.loss, l)
            assert g.shape == (0, 8) and g.dtype == dt
            loss, counts, slope = moe.balance(l, r.expert, mask)
            assert loss == 0 and not counts.any() and not slope.any()
            plan = moe.sort(r.expert, 8)
            assert plan.tokens == 0 and not plan.counts.any()


def test_block_of_nothing():
    """Norm, router and two grouped layers, under a gradient of a sum (strides 0)."""
    need_gpu()
    ln = norm.RMSNorm(256, device="cuda")
    up, down = (moe.GroupedLinear(4, *s, RECIPES[0], device="cuda") for s in ((256, 384), (384, 256)))
    x, stream = (torch.empty(0, 256, dtype=B, device="cuda", requires_grad=True) for _ in range(2))
    gate = torch.zeros(256, 4, dtype=B, device="cuda", requires_grad=True)
    n, total = ln(x, stream)
    r = moe.route((n @ gate).float(), 2)
    plan = moe.sort(r.expert, 4)
    y = total + moe.combine(down(torch.relu(up(n, plan, gather=True)), plan), plan, r.weights)
    (y.sum() + r.loss).backward()
    assert y.shape == x.grad.shape == stream.grad.shape == (0, 256)
    for p in (ln.weight, up.weight, down.weight, gate):
        assert p.grad.shape == p.shape and not p.grad.any()


@pytest.mark.parametrize("dt", [B, F])
def test_eps_of_zero(dt):
    """Rows that are not zero as always; a row of zeros has an infinite rstd, and NaN
    for y and for its codes, which are those of the cast."""
    need_gpu()
    x = torch.randn(5, 384, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda").to(dt)
    x[3] = 0
    y, _, rstd = norm.rms_norm_forward(x, eps=0.0)
    rows = [0, 1, 2, 4]
    t = x[rows].double()
    want = t * t.square().mean(1, keepdim=True) ** -0.5
    u = {B: 2.0 ** -8, F: 2.0 ** -24}[dt]
    assert ((y[rows].double() - want).abs() <= (u + 32 * 2.0 ** -24) * want.abs()).all()
    assert rstd[3] == float("inf") and y[3].isnan().all()
    dx, dw = norm.rms_norm_backward(torch.ones_like(x), x, None, rstd)
    assert dx[rows].isfinite().all() and dx[3].isnan().all() and dw.isnan().all()
    for recipe in (fm.BLOCK_1x128, fm.MX_1x32):
        q, _, r2 = norm.rms_norm_quantize(x, recipe, fm.E4M3, fm.ROW_AND_COL, eps=0.0)
        w = fm.quantize(x.float() * rstd[:, None], recipe, fm.E4M3, fm.ROW_AND_COL)
        assert torch.equal(r2, rstd) and torch.equal(q.q_row[:, :384], w.q_row[:, :384]) and torch.equal(q.q_col[:, :5], w.q_col[:, :5])
        assert torch.equal(q.s_row, w.s_row) and torch.equal(q.s_col, w.s_col)
