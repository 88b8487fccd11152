"""The RMS norm's backward pass has no more sets of weight sums than its workgroups
have rows for: 16 rows at a time of up to 256 columns, 4 of up to 1024, else one."""
import pytest

import fp8_scaled_quantization_scale_amd as fm


@pytest.mark.parametrize("cols,at_a_time", [(1, 16), (128, 16), (256, 16), (257, 4), (512, 4), (1000, 4), (1024, 4), (1025, 1), (4096, 1), (20000, 1)])
@pytest.mark.parametrize("rows", [0, 1, 3, 4, 5, 16, 17, 64, 127, 128, 129, 300, 1000, 1024, 1025, 5000, 1 << 20, 1 << 40])
def test_each_set_has_rows(rows, cols, at_a_time):
    sets, rest = divmod(fm.fp8_rms_norm_workspace(rows, cols), 4 * cols)
    assert rest == 0 and 1 <= sets <= max(1, -(-rows // at_a_time)) and sets <= 1024


@pytest.mark.parametrize("cols", [300, 512, 1024, 1025, 4096])
def test_enough_sets_to_fill_the_gpu(cols):
    assert fm.fp8_rms_norm_workspace(1 << 20, cols) == 512 * 4 * cols
    assert fm.fp8_rms_norm_workspace(128, cols) == (32 if cols <= 1024 else 128) * 4 * cols
