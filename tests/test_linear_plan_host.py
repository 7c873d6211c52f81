"""The plans of the 8-bit-integer products and the gated block, built with
AddressSanitizer and UndefinedBehaviorSanitizer and run by
tests/host_linear_plan_driver.cpp over sizes, CU counts and forced plans.  CPU
only: the plans are host arithmetic that needs no device."""

from __future__ import annotations

import os
import subprocess

import pytest

from tests.test_host_sanitizers import CLANG, CSRC, ROOT

DRIVER = os.path.join(ROOT, "tests", "host_linear_plan_driver.cpp")


@pytest.mark.skipif(not os.path.exists(CLANG), reason="ROCm toolchain not found")
def test_plans_keep_their_limits(tmp_path):
    exe = str(tmp_path / "plans")
    san = ["-fsanitize=address,undefined,float-cast-overflow", "-fno-sanitize-recover=all"]
    r = subprocess.run([CLANG, "-O1", "-g", "-std=c++17", *san, "-I", CSRC, DRIVER, "-o", exe], capture_output=True,
                       text=True)
    assert r.returncode == 0, r.stderr[-3000:]
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:abort_on_error=0:halt_on_error=1",
               UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1")
    r = subprocess.run([exe], capture_output=True, text=True, env=env, timeout=300)
    report = r.stdout + r.stderr
    assert r.returncode == 0, report[-4000:]
    assert "host plans ok" in r.stdout
    assert "runtime error" not in report and "AddressSanitizer" not in report, report[-4000:]
