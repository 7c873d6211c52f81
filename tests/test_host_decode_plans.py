"""Forced plans of the 4-bit product and the few-token expert layers, built with
AddressSanitizer and UndefinedBehaviorSanitizer and driven by
tests/host_decode_forced_driver.cpp, and what the layers set on their kernels
(tests/host_decode_lds_driver.cpp, on the built library).  CPU only."""

from __future__ import annotations

import os
import subprocess

import pytest

import moe_grouped_gemm_e4m3_amd as fg
from tests.test_host_decode import run
from tests.test_host_sanitizers import CLANG, CSRC, INCLUDE, ROCM, ROOT

SAN = ["-fsanitize=address,undefined,float-cast-overflow", "-fno-sanitize-recover=all"]


@pytest.mark.skipif(not os.path.exists(CLANG), reason="ROCm toolchain not found")
def test_forced_plans_fit_their_calls(tmp_path):
    exe = str(tmp_path / "forced")
    r = subprocess.run([CLANG, "-O1", "-g", "-std=c++17", *SAN, "-I", CSRC, os.path.join(ROOT, "tests", "host_decode_forced_driver.cpp"),
                        "-o", exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-3000:]
    run(exe, "host forced plans ok")


@pytest.mark.skipif(not os.path.exists(CLANG), reason="ROCm toolchain not found")
def test_a_kernels_lds_limit_does_not_depend_on_the_call(tmp_path):
    exe, lib = str(tmp_path / "lds"), os.path.abspath(fg.library_path())
    # the executable's own hipGetDevice and hipFuncSetAttribute come before the runtime's
    r = subprocess.run([CLANG, "-O1", "-g", "-std=c++17", "-rdynamic", "-D__HIP_PLATFORM_AMD__", "-I", INCLUDE, "-I", os.path.join(ROCM, "include"),
                        os.path.join(ROOT, "tests", "host_decode_lds_driver.cpp"), "-o", exe, lib, "-L", os.path.join(ROCM, "lib"),
                        "-lamdhip64", "-lpthread", "-Wl,-rpath," + os.path.dirname(lib) + ":" + os.path.join(ROCM, "lib")],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-3000:]
    run(exe, "host lds ok")
