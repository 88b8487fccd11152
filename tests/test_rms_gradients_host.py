"""The gradients that the RMS norm's autograd function hands to x and to the
residual have memory of their own wherever something may write to them: the
function on the CPU, with the formulas in torch in place of the kernels."""
import pytest
import torch

from fp8_scaled_quantization_scale_amd import norm

ROWS, COLS = 6, 8


@pytest.fixture(autouse=True)
def formulas(monkeypatch):
    def forward(x, weight=None, residual=None, eps=1e-6, stream=None):
        total = x if residual is None else x + residual
        rstd = (total.square().mean(1) + eps) ** -0.5
        return total * rstd[:, None] * weight, total, rstd

    def backward(dy, total, weight, rstd, dtotal=None, params=True, stream=None):
        n, g = total * rstd[:, None], dy * weight
        dx = rstd[:, None] * (g - n * (g * n).mean(1, keepdim=True))
        return dx if dtotal is None else dx + dtotal, (dy * n).sum(0) if params else None

    monkeypatch.setattr(norm, "rms_norm_forward", forward)
    monkeypatch.setattr(norm, "rms_norm_backward", backward)


class _Made(torch.autograd.Function):
    """Stands for a function of this package: its backward pass makes its own tensors."""

    @staticmethod
    def forward(ctx, x):
        return x.clone()

    @staticmethod
    def backward(ctx, d):
        return d * 1.0


_Made.__module__ = norm.__name__


def _leaf(*shape):
    return torch.randn(*shape, dtype=torch.float64).requires_grad_()


def _shares(a, b):
    return a.untyped_storage().data_ptr() == b.untyped_storage().data_ptr()


@pytest.mark.parametrize("outputs", ["both", "y", "total"])
@pytest.mark.parametrize("how", ["leaves", "views", "view and leaf", "made", "made and view", "sum of leaves", "made twice"])
def test_gradients_are_not_shared(how, outputs):
    torch.manual_seed(1)
    x, res = _leaf(2, 3, COLS), _leaf(2, 3, COLS)
    more = _leaf(2, 3, COLS)
    w = _leaf(COLS)
    rows = lambda t: t.reshape(-1, COLS)  # noqa: E731
    if how in ("leaves", "made twice"):
        x, res, more = (t.detach().reshape(ROWS, COLS).requires_grad_() for t in (x, res, more))
    dy, dtotal = torch.randn(ROWS, COLS, dtype=torch.float64), torch.randn(ROWS, COLS, dtype=torch.float64)

    def step():
        a, b = {"leaves": lambda: (x, res), "views": lambda: (rows(x), rows(res)), "view and leaf": lambda: (rows(x), rows(res * 1.0)),
                "made": lambda: (rows(_Made.apply(x)), rows(res)), "made and view": lambda: (rows(x), rows(_Made.apply(res))),
                "sum of leaves": lambda: (rows(x + more), rows(res)), "made twice": lambda: (_Made.apply(x), _Made.apply(res))}[how]()
        y, total = norm._RMSNormFn.apply(a, w, b, 1e-6)
        out = {"both": ([y, total], [dy, dtotal]), "y": ([y], [dy]), "total": ([total], [dtotal])}[outputs]
        torch.autograd.backward(*out)

    step()
    leaves = [x, res] + ([more] if how == "sum of leaves" else [])
    once = [t.grad.clone() for t in leaves]
    assert torch.equal(once[0], once[1]) and once[0].any()
    for i, t in enumerate(leaves):
        assert not any(_shares(t.grad, u.grad) for u in leaves[:i])
        assert not _shares(t.grad, dy) and not _shares(t.grad, dtotal)
    step()  # added in place
    for t, g in zip(leaves, once):
        assert torch.equal(t.grad, 2 * g)


def test_no_copy_where_a_backward_pass_of_the_package_reads_it():
    """(the residual stream between the package's layers costs no copy)"""
    x, res = _leaf(ROWS, COLS), _leaf(ROWS, COLS)
    made, other = _Made.apply(x), _Made.apply(res)
    view = made.view(3, 2, COLS).reshape(ROWS, COLS)
    for a, b in ((made, other), (view, other), (other, view), (made[:2], other), (made, made)):
        assert not norm._apart(a, b)
    for a in (x, x.view(-1), x * 1.0, made + res, made.detach().requires_grad_()):
        assert norm._apart(a, res) and norm._apart(a, x * 2.0) and norm._apart(a, other) and norm._apart(other, a)
    assert not norm._apart(x, None) and not norm._apart(x, res.detach())


def test_a_leaf_s_hook_does_not_reach_the_other_gradient():
    """A hook that scales a leaf's .grad as soon as it is there (an optimizer's step in
    the backward pass) while the other gradient has yet to be read."""
    torch.manual_seed(4)
    x, res, w = _leaf(2, 3, COLS), _leaf(ROWS, COLS), _leaf(COLS)

    def hook(t):
        t.grad.zero_()

    x.register_post_accumulate_grad_hook(hook)
    made = _Made.apply(res)
    y, total = norm._RMSNormFn.apply(x.reshape(ROWS, COLS), w, made, 1e-6)  # (what was made last goes first)
    dy, dtotal = torch.randn(ROWS, COLS, dtype=torch.float64), torch.randn(ROWS, COLS, dtype=torch.float64)
    torch.autograd.backward([y, total], [dy, dtotal])
    want, _ = norm.rms_norm_backward(dy, total.detach(), w.detach(), (total.detach().square().mean(1) + 1e-6) ** -0.5, dtotal)
    assert torch.equal(res.grad, want) and not x.grad.any()
