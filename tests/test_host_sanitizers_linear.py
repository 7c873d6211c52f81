"""The host code of the 8-bit-integer product and the gated block (argument
checks, plans, size arithmetic) built with AddressSanitizer and
UndefinedBehaviorSanitizer and driven by tests/host_linear_driver.cpp.  CPU
only; the device code is compiled as usual and never run here."""

from __future__ import annotations

import os
import subprocess

import pytest

from tests.test_host_sanitizers import CLANG, CSRC, HIPCC, HOST_SAN, INCLUDE, ROCM, ROOT

DRIVER = os.path.join(ROOT, "tests", "host_linear_driver.cpp")


@pytest.mark.skipif(not (os.path.exists(HIPCC) and os.path.exists(CLANG)), reason="ROCm toolchain not found")
def test_host_code_of_the_linear_operators(tmp_path):
    objs, jobs = [], []
    for src in ("fp8gemm.hip", "ue8m0.hip", "linear.hip"):
        objs.append(str(tmp_path / src.replace(".hip", ".o")))
        cmd = [HIPCC, "--offload-arch=gfx950", "-O1", "-g", "-std=c++17", "-fPIC",
               "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops", "-Wno-unused-command-line-argument",
               *HOST_SAN, "-I", INCLUDE, "-I", CSRC, "-c", os.path.join(CSRC, src), "-o", objs[-1]]
        jobs.append(subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True))
    for j in jobs:
        out, _ = j.communicate(timeout=600)
        assert j.returncode == 0, out[-3000:]
    exe = str(tmp_path / "host_linear_driver")
    san = ["-fsanitize=address,undefined", "-fno-sanitize-recover=all"]
    r = subprocess.run([CLANG, "-g", "-std=c++17", *san, "-I", INCLUDE, DRIVER, *objs,
                        "-L", os.path.join(ROCM, "lib"), "-lamdhip64", "-Wl,-rpath," + os.path.join(ROCM, "lib"),
                        "-o", exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-3000:]
    env = dict(os.environ, HIP_VISIBLE_DEVICES="",  # the host paths only, also on a machine with a GPU
               ASAN_OPTIONS="detect_leaks=0:abort_on_error=0:halt_on_error=1",
               UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1")
    r = subprocess.run([exe], capture_output=True, text=True, env=env, timeout=300)
    report = r.stdout + r.stderr
    assert r.returncode == 0, report[-4000:]
    assert "host linear ok" in r.stdout
    assert "runtime error" not in report and "AddressSanitizer" not in report, report[-4000:]
