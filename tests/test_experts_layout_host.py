"""fp8_gemm_grouped refuses experts' weight gradients that share elements, before
any GPU work."""
import pytest

import fp8_scaled_quantization_scale_amd as fm

P = 0x10000  # an aligned stand-in pointer, never dereferenced


def _call(m, n, experts, ldc, stride_c):
    return fm.fp8_gemm_grouped(P, fm.E4M3, P, 1152, P, fm.E4M3, P, 1152, 0, 0, 0, fm.GEMM_BLOCK_1x128_1x128,
                               fm.GROUP_CONTRACT, P, experts, 1152, m, n, 0, P, fm.OUT_BF16, ldc, stride_c, 0)


@pytest.mark.parametrize("ldc,stride_c", [
    (128, 0), (128, 64 * 128 - 1), (200, 63 * 200 + 127),  # the next begins before the last row's end
    (1024, 127), (1023, 128), (1024, 129), (8 * 200, 7 * 200),  # rows in turn, too close or past the next row
])
def test_shared_elements(ldc, stride_c):
    assert _call(64, 128, 8, ldc, stride_c) == fm.ERR_SHAPE
