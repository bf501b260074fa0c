"""The launches of the operators around the mixer, without a GPU: the library as built, its calls to the
runtime answered by a program that checks every launch (tests/launch/launch_driver.cpp)."""
import os
import shutil

import pytest

from gated_delta_rule_gdr_amd import library_path
from tests.test_sanitize_cpu import ROOT, _run


@pytest.mark.skipif(shutil.which("g++") is None or not os.path.isdir("/opt/rocm/include"),
                    reason="needs g++ and the ROCm headers")
def test_launches_fit_and_cover(tmp_path):
    exe = str(tmp_path / "launch")
    _run(["g++", "-std=c++17", "-O1", "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include", "-I", os.path.join(ROOT, "include"),
          "-I", os.path.join(ROOT, "gated_delta_rule_gdr_amd", "csrc"), os.path.join(ROOT, "tests", "launch", "launch_driver.cpp"),
          "-rdynamic", "-ldl", "-o", exe], ROOT)
    out = _run([exe, library_path()], ROOT)
    assert out.strip().startswith("ok"), out
