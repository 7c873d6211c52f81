"""Forced plans of the 4-bit product and the few-token expert layers, built with
AddressSanitizer and UndefinedBehaviorSanitizer and driven by
tests/host_decode_forced_driver.cpp.  CPU only."""

from __future__ import annotations

import os
import subprocess

import pytest

from tests.test_host_decode import run
from tests.test_host_sanitizers import CLANG, CSRC, ROOT

SAN = ["-fsanitize=address,undefined,float-cast-overflow", "-fno-sanitize-recover=all"]


@pytest.mark.skipif(not os.path.exists(CLANG), reason="ROCm toolchain not found")
def test_forced_plans_fit_their_calls(tmp_path):
    exe = str(tmp_path / "forced")
    r = subprocess.run([CLANG, "-O1", "-g", "-std=c++17", *SAN, "-I", CSRC, os.path.join(ROOT, "tests", "host_decode_forced_driver.cpp"),
                        "-o", exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-3000:]
    run(exe, "host forced plans ok")
