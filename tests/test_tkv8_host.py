"""The host half of libtkv under AddressSanitizer and UndefinedBehaviorSanitizer (CPU only), its part for the 8-bit cache,
rotations and windows: tests/sanitize/tkv8_host_driver.cpp."""
import os
import shutil
import subprocess

import pytest

from tests.test_host_sanitizers import ROCM, ROOT, SAN, _run


@pytest.mark.skipif(shutil.which("g++") is None or not os.path.exists(f"{ROCM}/include/hip"),
                    reason="g++ or the HIP headers not available")
def test_host_half_under_sanitizers(tmp_path):
    exe = str(tmp_path / "tkv8_host_driver")
    subprocess.run(["g++", "-std=c++17", *SAN, "-D__HIP_PLATFORM_AMD__", f"-I{ROCM}/include",
                    "-I" + os.path.join(ROOT, "include"),
                    os.path.join(ROOT, "tiled_tensor_bulk_amd", "csrc", "tkv_host.cpp"),
                    os.path.join(ROOT, "tests", "sanitize", "tkv8_host_driver.cpp"), "-o", exe],
                   check=True, capture_output=True)
    assert " 0 unexpected results" in _run(exe, tmp_path)
