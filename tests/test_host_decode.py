"""The host code of the router, the 4-bit cast and product and the few-token
expert layers (argument checks, plans, size arithmetic), built with
AddressSanitizer and UndefinedBehaviorSanitizer and driven by
tests/host_decode_driver.cpp and tests/host_decode_plan_driver.cpp.  CPU only; the
device code is compiled as usual and never run here."""

from __future__ import annotations

import os
import subprocess

import pytest

from tests.test_host_sanitizers import CLANG, CSRC, HIPCC, HOST_SAN, INCLUDE, ROCM, ROOT

ENV = dict(os.environ, HIP_VISIBLE_DEVICES="",  # the host paths only, also on a machine with a GPU
           ASAN_OPTIONS="detect_leaks=0:abort_on_error=0:halt_on_error=1", UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1")


def run(exe, said):
    r = subprocess.run([exe], capture_output=True, text=True, env=ENV, timeout=300)
    report = r.stdout + r.stderr
    assert r.returncode == 0, report[-4000:]
    assert said in r.stdout
    assert "runtime error" not in report and "AddressSanitizer" not in report, report[-4000:]


@pytest.mark.skipif(not os.path.exists(CLANG), reason="ROCm toolchain not found")
def test_plans_keep_their_limits(tmp_path):
    exe = str(tmp_path / "plans")
    san = ["-fsanitize=address,undefined,float-cast-overflow", "-fno-sanitize-recover=all"]
    r = subprocess.run([CLANG, "-O1", "-g", "-std=c++17", *san, "-I", CSRC, os.path.join(ROOT, "tests", "host_decode_plan_driver.cpp"),
                        "-o", exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-3000:]
    run(exe, "host plans ok")


@pytest.mark.skipif(not (os.path.exists(HIPCC) and os.path.exists(CLANG)), reason="ROCm toolchain not found")
def test_host_code_of_the_decode_operators(tmp_path):
    objs, jobs = [], []
    for src in ("fp8gemm.hip", "ue8m0.hip", "int4.hip", "experts.hip"):
        objs.append(str(tmp_path / src.replace(".hip", ".o")))
        cmd = [HIPCC, "--offload-arch=gfx950", "-O1", "-g", "-std=c++17", "-fPIC",
               "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops", "-Wno-unused-command-line-argument",
               *HOST_SAN, "-I", INCLUDE, "-I", CSRC, "-c", os.path.join(CSRC, src), "-o", objs[-1]]
        jobs.append(subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True))
    for j in jobs:
        out, _ = j.communicate(timeout=900)
        assert j.returncode == 0, out[-3000:]
    exe = str(tmp_path / "host_decode_driver")
    san = ["-fsanitize=address,undefined", "-fno-sanitize-recover=all"]
    r = subprocess.run([CLANG, "-g", "-std=c++17", *san, "-I", INCLUDE, os.path.join(ROOT, "tests", "host_decode_driver.cpp"), *objs,
                        "-L", os.path.join(ROCM, "lib"), "-lamdhip64", "-Wl,-rpath," + os.path.join(ROCM, "lib"),
                        "-o", exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-3000:]
    run(exe, "host decode ok")
