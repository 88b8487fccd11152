"""No kernel claims a larger alignment than its pointers have: the compiler's
front end (no code is made) finds no access through a type that is aligned to
more than the one it was taken from."""
import os
import subprocess

import pytest

from fp8_scaled_quantization_scale_amd import build

SOURCES = sorted(f for f in os.listdir(build.CSRC) if f.endswith(".hip"))


@pytest.mark.parametrize("source", SOURCES)
def test_front_end(source):
    try:
        hipcc = build.hipcc()
    except RuntimeError:
        pytest.skip("needs hipcc")
    r = subprocess.run([hipcc, *build._flags(), "--cuda-device-only", "-fsyntax-only", "-Werror=align-mismatch", "-x", "hip",
                        os.path.join(build.CSRC, source)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-3000:]
