"""The host layer of the block operators (include/ssmblock.h) built with
AddressSanitizer and UndefinedBehaviorSanitizer and run on the CPU: a driver
(``tests/sanitize/block_driver.cpp``) calls every entry point with buffers of exactly
their documented sizes over stand-ins for the runtime and the kernel launchers, which
read both ends of whatever their kernel would index.  Host code only."""
import os

from test_sanitizers import HERE, HIP_INCLUDE, ROOT, SAN, _build_and_run, _need

import pytest


def test_block_host_layer_under_asan_ubsan(tmp_path):
    _need("g++")
    if not os.path.isdir(os.path.join(HIP_INCLUDE, "hip")):
        pytest.skip("HIP headers not found")
    exe = str(tmp_path / "block_driver")
    csrc, here = os.path.join(ROOT, "sequence_scan_amd", "csrc"), os.path.join(HERE, "sanitize")
    _build_and_run(["g++", "-std=c++17", *SAN, "-D__HIP_PLATFORM_AMD__", f"-I{HIP_INCLUDE}",
                    os.path.join(csrc, "api.cpp"), os.path.join(csrc, "api_block.cpp"),
                    os.path.join(here, "fake_runtime.cpp"), os.path.join(here, "fake_block.cpp"),
                    os.path.join(here, "block_driver.cpp"), "-o", exe], exe, "block driver ok")
