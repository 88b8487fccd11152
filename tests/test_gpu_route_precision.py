"""The router's probabilities, weights and gradient keep binary32's precision far
below the largest logit: no error grows with the distance.

The logits are multiples of 1/64, so that their differences are exact.  Steps of
2^-24 (half a step of binary32): a weight's or a gradient's exponential is off by at
most 2 by the hardware's own last place and 0.35 by its argument's two roundings
(each at most 2^-26 of a number below 1/2, times ln 2): EXP = 2.4.  A sum of
positive terms over the experts adds, at most, a lane's experts and six steps across
the lanes: ADDS.  A weight is a quotient of two such: 2 EXP + ADDS + 1.  A
probability in the gradient is a product with a rounded reciprocal: P = 2 EXP + ADDS
+ 2; p (slope dloss - dot) then has terms whose own errors are at most 2 P + ADDS +
4.  What lies below 2^-126 is off by two units of 2^-149 more."""
import pytest
import torch

from fp8_scaled_quantization_scale_amd import moe
from gpu_util import need_gpu

pytestmark = pytest.mark.gpu

E32 = 2.0 ** -24
EXP, DENORMAL = 2.4, 2.0 ** -148
U = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
B, F = torch.bfloat16, torch.float32


def _adds(experts):
    lanes, v = (16 if experts <= 256 else 64), 1
    while lanes * v < experts:
        v *= 2
    return v + 6


def _logits(tokens, experts, dt, least, seed=0):
    """Multiples of 1/64 from `least` to 0 (BF16: of 1, which it holds), with a 0 in each row."""
    g = torch.Generator(device="cuda").manual_seed(seed + experts)
    step = 1 if dt == B else 64
    x = torch.randint(least * step, 1, (tokens, experts), generator=g, device="cuda").double() / step
    x[torch.arange(tokens, device="cuda"), torch.randint(0, experts, (tokens,), generator=g, device="cuda")] = 0.0
    assert torch.equal(x.to(dt).double(), x)
    return x.to(dt), g


@pytest.mark.parametrize("normalize", [False, True])
@pytest.mark.parametrize("experts,topk,dt", [(2, 2, F), (8, 8, F), (8, 8, B), (16, 16, F), (64, 16, F), (64, 33, F), (256, 16, F), (100, 100, F),
                                             (512, 16, F), (1000, 70, B)])
def test_weights(experts, topk, dt, normalize):
    need_gpu()
    for least in (-10, -80, -100):
        l, _ = _logits(700, experts, dt, least)
        r = moe.route(l, topk, normalize)
        at = r.expert.long()
        p = torch.softmax(l.double(), 1).gather(1, at)
        if normalize:
            p = p / p.sum(1, keepdim=True)
        off = (r.weights.double() - p).abs() - ((2 * EXP + _adds(experts) + 1) * E32 * p + DENORMAL)
        assert not (off > 0).any(), f"{int((off > 0).sum())} weights, the worst {((r.weights.double() / p - 1).abs().max() / E32).item():.1f} half steps"


@pytest.mark.parametrize("weights", [False, True])
@pytest.mark.parametrize("experts,topk,dt", [(2, 2, F), (8, 2, F), (8, 8, F), (16, 4, F), (64, 8, F), (256, 8, F), (300, 80, F), (8, 2, B)])
def test_gradient(experts, topk, dt, weights):
    need_gpu()
    l, g = _logits(500, experts, dt, -80, 1)
    r = moe.route(l, topk, False)
    at = r.expert.long()
    slope, dloss = torch.randn(experts, generator=g, device="cuda"), torch.tensor(0.7, device="cuda")
    dw = torch.randn(500, topk, generator=g, device="cuda") if weights else None
    got = moe.route_backward(l, r.expert, dw, slope, dloss, normalize=False)
    p = torch.softmax(l.double(), 1)
    dp = (slope * dloss).double()[None].expand_as(p)  # (the product's rounding is the kernel's)
    size = dp.abs()
    if weights:
        dp, size = dp.scatter_add(1, at, dw.double()), size.scatter_add(1, at, dw.double().abs())
    ref = p * (dp - (p * dp).sum(1, keepdim=True))
    size = p * (size + (p * size).sum(1, keepdim=True))
    adds = _adds(experts)
    tol = (2 * (2 * EXP + adds + 2) + adds + 4) * E32 * size + U[dt] * ref.abs() + 2 * DENORMAL
    bad = (got.double() - ref).abs() > tol
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()}"


@pytest.mark.parametrize("dt", [B, F])
def test_loss_of_choices_far_below(dt):
    """One token, whose choice is not its largest logit: the loss is 2 p of it, and
    its slope's and product's roundings (4) come on top."""
    need_gpu()
    expert = torch.tensor([[1]], dtype=torch.int32, device="cuda")
    for d in range(-80 * 64, -40 * 64, 64 if dt == B else 23):
        l = torch.tensor([[0.0, d / 64]], device="cuda").to(dt)
        loss, _, _ = moe.balance(l, expert)
        want = 2.0 * torch.softmax(l.double(), 1)[0, 1].item()
        assert abs(loss.item() - want) <= (2 * EXP + _adds(2) + 2 + 4) * E32 * want, d


@pytest.mark.parametrize("far", [4, 12, 30])
@pytest.mark.parametrize("experts,topk", [(2, 2), (8, 2), (8, 8), (64, 8), (64, 40), (256, 16), (300, 8), (300, 100)])
def test_normalized_weights_where_one_expert_has_nearly_all(experts, topk, far):
    """dl = w (dw - c), c = <w, dw>, where dw - c is small for the expert whose weight
    is near 1.  A weight is off by W = 2 EXP + ADDS + 2 steps, the mean of dw - c that
    is taken out at the end by 2 W + ADDS + 6 of the mean of |dw - c|; what c itself is
    off by enters by its rounding alone, a step of a step of |dw|."""
    need_gpu()
    g = torch.Generator(device="cuda").manual_seed(experts + far)
    l = -far - torch.randint(0, 10 * 64, (400, experts), generator=g, device="cuda").double() / 64
    l[torch.arange(400, device="cuda"), torch.randint(0, experts, (400,), generator=g, device="cuda")] = 0.0
    l = l.float()
    r = moe.route(l, topk, True)
    dw = torch.randn(400, topk, generator=g, device="cuda")
    got = moe.route_backward(l, r.expert, dw, r.slope, None, normalize=True)
    at = r.expert.long()
    w = torch.softmax(l.double().gather(1, at), 1)
    off = dw.double() - (w * dw.double()).sum(1, keepdim=True)
    off = off - (w * off).sum(1, keepdim=True)  # (64 bits have the same trouble)
    adds = _adds(experts) + -(-topk // 16)
    c = 2 * (2 * EXP + adds + 2) + adds + 6
    tol = w * (c * E32 * (off.abs() + (w * off.abs()).sum(1, keepdim=True)) + (c * E32) ** 2 * dw.abs().amax(1, keepdim=True)) + 2 * DENORMAL
    bad = (got.double().gather(1, at) - w * off).abs() > tol
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()}"


@pytest.mark.parametrize("dt", [F, B])
@pytest.mark.parametrize("experts", [1, 2, 7, 16, 64, 256, 300, 1000])
def test_loss_gradient_with_even_loads(experts, dt):
    """p (s - <p, s>), s = slope dloss: what all slopes have in common has no gradient.
    Equal slopes give zeros; slopes that differ by steps of 2^-22 of themselves (their
    differences are exact) an error in proportion to the differences, P and ADDS as above."""
    need_gpu()
    l, g = _logits(300, experts, dt, -12, 2)
    dloss = torch.tensor(0.3, device="cuda")
    slope = torch.full((experts,), 1.7, device="cuda")
    assert not moe.route_backward(l, None, None, slope, dloss).any()
    over = torch.randint(0, 64, (experts,), generator=g, device="cuda").float() * 2.0 ** -22
    slope = 1.5 + over
    assert torch.equal(slope.double() - 1.5, over.double())
    got = moe.route_backward(l, None, None, slope, dloss)
    s = (slope.double() - slope.double().min()) * dloss.double()
    p = torch.softmax(l.double(), 1)
    ref = p * (s - (p * s).sum(1, keepdim=True))
    size = p * (s + (p * s).sum(1, keepdim=True))
    adds = _adds(experts)
    tol = (2 * (2 * EXP + adds + 2) + adds + 4) * E32 * size + U[dt] * ref.abs()
    assert ((got.double() - ref).abs() <= tol).all()


def test_loss_gradient_of_even_routing():
    """Each expert chosen as often: the loss has no gradient, to the bit."""
    need_gpu()
    l = torch.randn(64, 8, device="cuda").requires_grad_()
    expert = (torch.arange(64, device="cuda")[:, None] + torch.arange(2, device="cuda")).remainder(8)
    loss, counts, _ = moe.balance(l, expert)
    assert (counts == 16).all()
    loss.backward()
    assert not l.grad.any()
