"""Host sanitizer build (CPU only) of the layer norm's and the experts' argument
validation (csrc/api_norm.cpp, csrc/api_moe.cpp, the launchers replaced by
recording stubs), driven over edge inputs by tests/sanitize/
abi_operators_driver.cpp.  Any report aborts the program
(-fno-sanitize-recover=all), so a zero exit means none was raised."""
import os
import shutil

import pytest

from test_sanitize import HERE, ROOT, SAN, _build_and_run


@pytest.mark.skipif(shutil.which("g++") is None or not os.path.isdir("/opt/rocm/include"),
                    reason="needs g++ and the ROCm headers")
def test_operator_validation_under_sanitizers(tmp_path):
    exe = str(tmp_path / "abi_operators_driver")
    csrc = os.path.join(ROOT, "fp8_scaled_quantization_scale_amd", "csrc")
    sources = [os.path.join(csrc, "api_norm.cpp"), os.path.join(csrc, "api_moe.cpp"), os.path.join(HERE, "abi_operators_driver.cpp")]
    cmd = (["g++", "-std=c++17"] + SAN + ["-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include", "-I" + os.path.join(ROOT, "include"),
                                           "-I" + csrc] + sources + ["-o", exe])
    assert "operator validation ok" in _build_and_run(cmd, exe)
