"""The RMS norm's statistics lose no more to rounding than torch's own FP32
reduction does.

Over the rows of one input the error of rstd against 64 bits is a root mean square
over many independent roundings; of 4096 rows it is known to 1 / sqrt(2 * 4096) =
1.1%, and the ratio of two such to 1.6%: 5% is three times that.  Rows of one FP32
value make each partial sum exact but for the square's rounding where the sums are
taken in pairs and the width is a power of two that fills the threads: then rstd is
off by half a step for the square (its root halves it), one for the root and one for
the quotient, in steps of 2^-24."""
import pytest
import torch

from fp8_scaled_quantization_scale_amd import norm
from gpu_util import need_gpu

pytestmark = pytest.mark.gpu

E32 = 2.0 ** -24


@pytest.mark.parametrize("cols", [512, 1024, 4096, 5120, 6144, 7168, 8192, 16384, 40000])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_rstd_as_near_as_torch(cols, dt):
    need_gpu()
    g = torch.Generator(device="cuda").manual_seed(cols)
    x = torch.randn(4096, cols, generator=g, device="cuda").to(dt)
    exact = torch.cat([(c.double().square().mean(1) + 1e-6) ** -0.5 for c in x.split(512)])
    plain = torch.cat([1.0 / torch.sqrt((c.float() * c.float()).mean(1) + 1e-6) for c in x.split(512)])
    _, _, rstd = norm.rms_norm_forward(x)
    rms = lambda r: (r.double() / exact - 1).square().mean().sqrt().item() / E32  # noqa: E731
    assert rms(rstd) <= 1.05 * rms(plain), (rms(rstd), rms(plain))


@pytest.mark.parametrize("cols", [128, 256, 512, 1024, 2048, 4096, 8192, 16384])
def test_rows_of_one_value(cols):
    need_gpu()
    g = torch.Generator(device="cuda").manual_seed(cols + 1)
    v = torch.rand(2000, 1, generator=g, device="cuda") + 0.5
    _, _, rstd = norm.rms_norm_forward(v.expand(2000, cols).contiguous(), eps=0.0)
    assert ((rstd.double() * v[:, 0].double() - 1).abs() <= 2.51 * E32).all()
