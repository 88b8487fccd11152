"""Host sanitizer build (CPU only) of the RMS norm's and the router's argument
validation (csrc/api_rms.cpp, csrc/api_route.cpp, the launchers replaced by
recording stubs), driven over edge inputs by tests/sanitize/
abi_rms_route_driver.cpp.  Any report aborts the program
(-fno-sanitize-recover=all), so a zero exit means none was raised."""
import os
import shutil

import pytest

from test_sanitize import HERE, ROOT, SAN, _build_and_run


@pytest.mark.skipif(shutil.which("g++") is None or not os.path.isdir("/opt/rocm/include"),
                    reason="needs g++ and the ROCm headers")
def test_rms_and_route_validation_under_sanitizers(tmp_path):
    exe = str(tmp_path / "abi_rms_route_driver")
    csrc = os.path.join(ROOT, "fp8_scaled_quantization_scale_amd", "csrc")
    sources = [os.path.join(csrc, "api_rms.cpp"), os.path.join(csrc, "api_route.cpp"), os.path.join(HERE, "abi_rms_route_driver.cpp")]
    cmd = (["g++", "-std=c++17"] + SAN + ["-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include", "-I" + os.path.join(ROOT, "include"),
                                           "-I" + csrc] + sources + ["-o", exe])
    assert "rms and route validation ok" in _build_and_run(cmd, exe)
