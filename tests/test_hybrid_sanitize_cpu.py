"""Host validation and size arithmetic of the RMS norm, linear attention with a decay and the paged cache
(gdr2_hybrid_api.hip, compiled as plain C++ against launch stand-ins) under AddressSanitizer and
UndefinedBehaviorSanitizer."""
import os
import shutil

import pytest

from tests.test_sanitize_cpu import ROOT, SAN, _run


@pytest.mark.skipif(shutil.which("g++") is None or not os.path.isdir("/opt/rocm/include"),
                    reason="needs g++ and the ROCm headers")
def test_hybrid_abi_under_sanitizers(tmp_path):
    exe = str(tmp_path / "hybrid_san")
    csrc = os.path.join(ROOT, "gated_delta_rule_gdr_amd", "csrc")
    _run(["g++", "-std=c++17", "-x", "c++", "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include",
          "-I", os.path.join(ROOT, "include"), "-I", csrc, *SAN, os.path.join(csrc, "gdr2_hybrid_api.hip"),
          os.path.join(ROOT, "tests", "sanitize", "hybrid_driver.cpp"), "-o", exe], ROOT)
    out = _run([exe], ROOT)
    assert out.strip().startswith("ok"), out
