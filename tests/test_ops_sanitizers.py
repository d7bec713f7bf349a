"""The operators' argument checks, tensor lists and launches under
AddressSanitizer and UndefinedBehaviorSanitizer (CPU): ops_abi.cpp, abi.cpp and
plan.cpp built with g++ against a driver that records launches."""
import os
import shutil

import pytest

from tests.test_host_sanitizers import ROOT, SAN, _run


@pytest.mark.skipif(shutil.which("g++") is None or not os.path.isdir("/opt/rocm/include"), reason="needs g++ and the HIP headers")
def test_operators_abi_under_sanitizers(tmp_path):
    csrc = os.path.join(ROOT, "blockwise_fp8_zero_amd", "csrc")
    exe = str(tmp_path / "ops_driver")
    out = _run(["g++", "-std=c++17", *SAN, "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include", "-I" + os.path.join(ROOT, "include"),
                "-I" + csrc, os.path.join(csrc, "plan.cpp"), os.path.join(csrc, "abi.cpp"), os.path.join(csrc, "ops_abi.cpp"),
                os.path.join(ROOT, "tests", "sanitize", "ops_driver.cpp"), "-o", exe], exe)
    assert "all checks passed" in out
