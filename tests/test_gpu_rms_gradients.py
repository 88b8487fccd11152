"""RMSNorm's and RMSNormLinear's gradients of x and of the residual do not share
memory where they become the .grad of leaves: a second backward pass adds to each
once, and writing to one leaves the other."""
import pytest
import torch

from fp8_scaled_quantization_scale_amd import linear, norm
from gpu_util import need_gpu

pytestmark = pytest.mark.gpu


def _layers():
    return {"norm": norm.RMSNorm(256, device="cuda"),
            "linear": linear.RMSNormLinear(256, 128, recipe=linear.Float8BlockScaling(), device="cuda")}


@pytest.mark.parametrize("which", ["norm", "linear"])
@pytest.mark.parametrize("outputs", [(0, 1), (0,), (1,)])
@pytest.mark.parametrize("shape", [(64, 256), (4, 16, 256)])
def test_leaves(which, outputs, shape):
    need_gpu()
    torch.manual_seed(2)
    layer = _layers()[which]
    x, res = (torch.randn(shape, device="cuda").bfloat16().requires_grad_() for _ in range(2))
    d = None

    def step():
        nonlocal d
        out = layer(x, res)
        d = d or [torch.randn_like(t) for t in out]
        torch.autograd.backward([out[i] for i in outputs], [d[i] for i in outputs])

    step()
    assert torch.equal(x.grad, res.grad) and x.grad.any()
    once = x.grad.clone()
    step()
    assert torch.equal(x.grad, 2 * once) and torch.equal(res.grad, 2 * once)
    x.grad.zero_()
    assert torch.equal(res.grad, 2 * once) and all(t.grad is None or t.grad.data_ptr() != x.grad.data_ptr() for t in (*d, res))


@pytest.mark.parametrize("which", ["norm", "linear"])
@pytest.mark.parametrize("leaf", [False, True])
def test_behind_layers(which, leaf):
    """x from a layer of the package, the residual from another, when no copy is made,
    or a leaf: the gradients are those of the two by themselves."""
    need_gpu()
    torch.manual_seed(3)
    layer, before = _layers()[which], linear.Linear(128, 256, recipe=linear.Float8BlockScaling(), device="cuda")
    first = norm.RMSNorm(256, device="cuda")
    a, res = torch.randn(4, 16, 128, device="cuda").bfloat16().requires_grad_(), torch.randn(4, 16, 256, device="cuda").bfloat16().requires_grad_()
    x, stream = before(a), res if leaf else first(res)
    assert norm._apart(norm._rows_of(x, 256), norm._rows_of(stream, 256)) == leaf
    alone = [t.detach().requires_grad_() for t in (x, stream)]
    y, total = layer(*alone)
    dy = torch.randn_like(y)
    torch.autograd.backward([y, total], [dy, torch.ones_like(total)])
    y, total = layer(x, stream)
    torch.autograd.backward([y, total], [dy, torch.ones_like(total)])
    want, = torch.autograd.grad(before(a), a, alone[0].grad)
    assert torch.equal(a.grad, want)
    want = alone[1].grad if leaf else torch.autograd.grad(first(res), res, alone[1].grad)[0]
    assert torch.equal(res.grad, want)
