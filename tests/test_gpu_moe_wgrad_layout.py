"""Weight gradients whose experts' rows lie in turn ([M x experts x N] in
memory), and the refusal of products that share elements."""
import pytest
import torch

import fp8_scaled_quantization_scale_amd as fm
from fp8_scaled_quantization_scale_amd import moe
from gpu_util import need_gpu

pytestmark = pytest.mark.gpu


def _operands(m, n, rows):
    g = torch.Generator(device="cuda").manual_seed(7)
    codes = lambda r: torch.randint(0, 0x70, (r, rows), generator=g, device="cuda", dtype=torch.uint8)  # noqa: E731
    scales = lambda r: torch.rand(r, rows // 128, generator=g, device="cuda") + 0.5  # noqa: E731
    return codes(m), scales(m), codes(n), scales(n)


@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("m,n,experts,gap", [(300, 264, 3, 0), (1, 40, 5, 0), (64, 100, 4, 13), (256, 128, 1, 0)])
def test_rows_in_turn(m, n, experts, gap, out):
    need_gpu()
    rows = 128 * (experts + 1)
    a, s_a, b, s_b = _operands(m, n, rows)
    offsets = torch.arange(experts + 1, dtype=torch.int32, device="cuda") * 128
    want = moe.gemm_wgrad(a, fm.E4M3, s_a, b, fm.E4M3, s_b, fm.GEMM_BLOCK_1x128_1x128, offsets, out)
    buf = torch.full((m, experts, n + gap), 7.0, dtype=out, device="cuda")
    c = buf[..., :n].permute(1, 0, 2)
    got = moe.gemm_wgrad(a, fm.E4M3, s_a, b, fm.E4M3, s_b, fm.GEMM_BLOCK_1x128_1x128, offsets, c=c)
    assert got is c and torch.equal(got, want) and (buf[..., n:] == 7).all()


def test_shared_elements_are_refused():
    need_gpu()
    a, s_a, b, s_b = _operands(64, 32, 512)
    offsets = torch.tensor([0, 128, 256], dtype=torch.int32, device="cuda")
    buf = torch.zeros(4096 * 4, device="cuda")
    for strides in ((0, 32, 1), (32 * 63, 32, 1), (31, 64, 1), (32, 63, 1), (64 * 62, 64, 1)):
        with pytest.raises(fm.Fp8Error):
            moe.gemm_wgrad(a, fm.E4M3, s_a, b, fm.E4M3, s_b, fm.GEMM_BLOCK_1x128_1x128, offsets,
                           c=buf.as_strided((2, 64, 32), strides))
