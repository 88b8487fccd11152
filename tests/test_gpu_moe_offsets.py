"""Grouped products under an offsets array that falls somewhere: a bound below
an earlier one is raised to it, so that no row belongs to two experts and every
tile lies in the buffers.  Bit for bit the products of the array with these
bounds raised by hand."""
import pytest
import torch

import fp8_scaled_quantization_scale_amd as fm
from fp8_scaled_quantization_scale_amd import moe
from gpu_util import need_gpu

pytestmark = pytest.mark.gpu


def _case(shape, mx, seed):
    """codes of finite values and scales along the last dimension"""
    g = torch.Generator(device="cuda").manual_seed(seed)
    codes = torch.randint(0, 0x70, shape, generator=g, device="cuda", dtype=torch.uint8)
    per = shape[-1] // (32 if mx else 128)
    if mx:
        return codes, torch.randint(120, 130, (*shape[:-1], per), generator=g, device="cuda", dtype=torch.uint8)
    return codes, torch.rand(*shape[:-1], per, generator=g, device="cuda") + 0.5


def _raised(offsets, rows):
    out, top = [], 0
    for v in offsets:
        top = max(top, min(max(v, 0), rows) // 128 * 128)
        out.append(top)
    return out


def _both(call, offsets, rows, c):
    """call(offsets, c) on the array as it is and on the raised one, into equal buffers"""
    a, b = c, c.clone()
    call(torch.tensor(offsets, dtype=torch.int32, device="cuda"), a)
    call(torch.tensor(_raised(offsets, rows), dtype=torch.int32, device="cuda"), b)
    assert torch.equal(a, b)
    return a


# large tiles and small ones (1664 rows), bounds that fall once, to nothing, twice, and
# a first expert without rows whose bound is not 0
@pytest.mark.parametrize("rows,offsets", [
    (16384, [0, 9000, 4000, 12000, 16384]), (16384, [16384, 0, 5000, 2560, 1 << 30]), (16384, [256, 16000, 100, 15000, 90]),
    (1664, [0, 900, 400, 1200, 1664]), (1664, [256, 1600, 100, 1500, -7]),
    (16384, [300, 200, 9000, 100, 16384]), (1664, [300, 200, 1500, 100, 1664])])
@pytest.mark.parametrize("mx", [False, True], ids=["block", "mx"])
def test_rows(rows, offsets, mx):
    need_gpu()
    n, k, experts = 640, 512, 4
    a, s_a = _case((rows, k), mx, 1)
    b, s_b = _case((experts, n, k), mx, 2)
    if not mx:
        s_b = s_b[:, ::128].contiguous()
    recipe = fm.GEMM_MX_1x32 if mx else fm.GEMM_BLOCK_1x128_128x128
    c = torch.full((rows, n), 7.0, device="cuda")
    c = _both(lambda o, c: moe.gemm(a, fm.E4M3, s_a, b, fm.E4M3, s_b, recipe, o, c=c), offsets, rows, c)
    first, last = _raised(offsets, rows)[0], _raised(offsets, rows)[-1]
    assert (c[:first] == 7).all() and (c[last:] == 7).all() and not (c[first:last] == 7).all(1).any()


@pytest.mark.parametrize("offsets", [[0, 1300, 600, 1800, 2048], [2048, 0, 900, 300, 1 << 30], [256, 2000, 100, 1500, -7]])
@pytest.mark.parametrize("mx", [False, True], ids=["block", "mx"])
def test_contraction(offsets, mx):
    need_gpu()
    rows, m, n = 2048, 200, 328
    a, s_a = _case((m, rows), mx, 3)
    b, s_b = _case((n, rows), mx, 4)
    recipe = fm.GEMM_MX_1x32 if mx else fm.GEMM_BLOCK_1x128_1x128
    c = torch.full((4, m, n), 7.0, device="cuda")
    c = _both(lambda o, c: moe.gemm_wgrad(a, fm.E4M3, s_a, b, fm.E4M3, s_b, recipe, o, c=c), offsets, rows, c)
    r = _raised(offsets, rows)
    for e in range(4):
        assert c[e].any() == (r[e] < r[e + 1])


def test_the_most_experts_and_all_rows_in_every_other():
    """1024 bounds that jump between no rows and all: the first expert has them all."""
    need_gpu()
    rows, n, k, experts = 270080, 256, 128, 1024
    a, s_a = _case((rows, k), False, 5)
    b, s_b = _case((experts, n, k), False, 6)
    s_b = s_b[:, ::128].contiguous()
    c = torch.zeros(rows, n, dtype=torch.bfloat16, device="cuda")
    offsets = [0] + [rows if e % 2 == 0 else 0 for e in range(experts)]
    c = _both(lambda o, c: moe.gemm(a, fm.E4M3, s_a, b, fm.E4M3, s_b, fm.GEMM_BLOCK_1x128_128x128, o, c=c), offsets, rows, c)
    want = fm.gemm(a, fm.E4M3, s_a, b[0], fm.E4M3, s_b[0].contiguous(), fm.GEMM_BLOCK_1x128_128x128, k)
    assert torch.equal(c, want)
