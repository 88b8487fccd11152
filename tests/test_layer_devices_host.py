"""The layers make their calls with the input's device current, whichever device
the caller left current: casts and products are launched on the current device's
stream.  Tensors of another device than the input's are refused.  (Stand-ins for
tensors on a second GPU; no call reaches the library.)"""
import types

import pytest
import torch

import fp8_scaled_quantization_scale_amd as fm
from fp8_scaled_quantization_scale_amd import linear, moe

ONE, ZERO = torch.device("cuda", 1), torch.device("cuda", 0)


class _On:
    """A tensor on `device`, as far as a layer's forward looks at it."""
    is_cuda, dtype, requires_grad = True, torch.bfloat16, False

    def __init__(self, device, *shape):
        self.device, self.shape = device, shape

    def dim(self):
        return len(self.shape)

    def stride(self, i=None):
        return (self.shape[1], 1)[i]

    def numel(self):
        return 1

    def reshape(self, *_):
        return self

    contiguous = view = reshape


class _Scopes:
    """Stands for _scope: which devices' scopes are open."""

    def __init__(self):
        self.open = []

    def __call__(self, device, stream):
        assert stream is None
        scopes = self

        class _One:
            def __enter__(self):
                scopes.open.append(device)

            def __exit__(self, *_):
                scopes.open.pop()
        return _One()


@pytest.fixture
def scopes(monkeypatch):
    s = _Scopes()
    monkeypatch.setattr(linear, "_scope", s, raising=False)
    monkeypatch.setattr(moe, "_scope", s)
    monkeypatch.setattr(linear, "load", lambda: None)
    return s


def _case(which, device_of_weight=ONE):
    rec = linear.Float8BlockScaling()
    x = _On(ONE, 128, 128)
    if which == "Linear":
        layer, fn, args = linear.Linear(128, 128, recipe=rec), (linear, "_Fp8LinearFn"), (x,)
    elif which == "RMSNormLinear":
        layer, fn, args = linear.RMSNormLinear(128, 128, recipe=rec), (linear, "_RmsNormLinearFn"), (x,)
        layer._parameters["norm_weight"] = _On(ONE, 128)
    else:
        layer, fn = moe.GroupedLinear(2, 128, 128, rec), (moe, "_GroupedLinearFn")
        args = (x, types.SimpleNamespace(experts=2, rows=256, offsets=_On(ONE, 3)))
    layer._parameters["weight"] = _On(device_of_weight, 128, 128)
    return layer, fn, args


@pytest.mark.parametrize("which", ["Linear", "RMSNormLinear", "GroupedLinear"])
def test_calls_run_on_the_input_s_device(which, scopes, monkeypatch):
    layer, (module, name), args = _case(which)
    seen = []

    def apply(*_):
        seen.append(list(scopes.open))
        return _On(ONE, 128, 128)

    monkeypatch.setattr(module, name, types.SimpleNamespace(apply=apply))
    layer(*args)
    assert seen == [[ONE]] and not scopes.open


@pytest.mark.parametrize("which", ["Linear", "RMSNormLinear", "GroupedLinear"])
def test_a_weight_on_another_device_is_refused(which, scopes):
    layer, _, args = _case(which, ZERO)
    with pytest.raises(fm.Fp8Error, match="one device"):
        layer(*args)


def test_norm_weight_on_another_device_is_refused(scopes):
    layer, _, args = _case("RMSNormLinear")
    layer._parameters["norm_weight"] = _On(ZERO, 128)
    with pytest.raises(fm.Fp8Error, match="one device"):
        layer(*args)
