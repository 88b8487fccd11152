"""fp8_quantize's channel recipe refuses sizes whose launches would be cut: a
launch counts its work-items modulo 2^32, which are 256 per 128 x 128 tile, and
16 per row (column) where that has several tiles.  Refusals only, before any GPU
work."""
import pytest

import fp8_scaled_quantization_scale_amd as fm

P = 0x10000  # an aligned stand-in pointer, never dereferenced


def _call(rows, cols, orient):
    ld_r, ld_c = (cols + 15) // 16 * 16, (rows + 15) // 16 * 16
    return fm.fp8_quantize(P, fm.IN_BF16, rows, cols, ld_r, fm.CHANNEL, fm.E4M3, orient, 0, P, ld_r, P, P, ld_c, P, None, None,
                           None, None, 0)


@pytest.mark.parametrize("rows,cols,orient", [
    (1 << 31, 128, fm.ROW), (128, 1 << 31, fm.COL), ((1 << 30) + 128, 256, fm.ROW), (1 << 19, 1 << 19, fm.ROW_AND_COL),  # 2^24 tiles
    ((1 << 28) - 15, 129, fm.ROW), ((1 << 28) - 15, 136, fm.ROW_AND_COL), (129, (1 << 28) - 15, fm.COL),
])
def test_refused(rows, cols, orient):
    assert _call(rows, cols, orient) == fm.ERR_UNSUPPORTED
