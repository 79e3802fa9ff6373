"""The host layer of the model operators (include/ssmmodel.h), with the plans of their tiles,
pieces and workspaces, built with AddressSanitizer and UndefinedBehaviorSanitizer and run
on the CPU (``tests/sanitize/model_driver.cpp``).  Host code only."""
import os

from test_sanitizers import HERE, HIP_INCLUDE, ROOT, SAN, _build_and_run, _need

import pytest


def test_model_host_layer_under_asan_ubsan(tmp_path):
    _need("g++")
    if not os.path.isdir(os.path.join(HIP_INCLUDE, "hip")):
        pytest.skip("HIP headers not found")
    exe = str(tmp_path / "model_driver")
    csrc, here = os.path.join(ROOT, "sequence_scan_amd", "csrc"), os.path.join(HERE, "sanitize")
    _build_and_run(["g++", "-std=c++17", *SAN, "-D__HIP_PLATFORM_AMD__", f"-I{HIP_INCLUDE}",
                    *[os.path.join(csrc, f) for f in ("api.cpp", "api_block.cpp", "api_model.cpp")],
                    *[os.path.join(here, f) for f in ("fake_runtime.cpp", "fake_block.cpp", "fake_model.cpp", "model_driver.cpp")],
                    "-o", exe], exe, "model driver ok")
