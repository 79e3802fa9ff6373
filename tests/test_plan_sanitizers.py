"""Plans at the ends of their range through the sanitised host layer on the CPU
(``tests/sanitize/plan_driver.cpp``): neither their arithmetic nor what it launches may overflow."""
import os

from test_sanitizers import HERE, HIP_INCLUDE, ROOT, SAN, _build_and_run, _need

import pytest


def test_longest_time_chunks(tmp_path):
    _need("g++")
    if not os.path.isdir(os.path.join(HIP_INCLUDE, "hip")):
        pytest.skip("HIP headers not found")
    exe = str(tmp_path / "plan_driver")
    csrc, here = os.path.join(ROOT, "sequence_scan_amd", "csrc"), os.path.join(HERE, "sanitize")
    _build_and_run(["g++", "-std=c++17", *SAN, "-D__HIP_PLATFORM_AMD__", f"-I{HIP_INCLUDE}",
                    os.path.join(csrc, "api.cpp"), os.path.join(csrc, "api_block.cpp"),
                    os.path.join(here, "fake_runtime.cpp"), os.path.join(here, "fake_block.cpp"),
                    os.path.join(here, "plan_driver.cpp"), "-o", exe], exe, "plan driver ok")
