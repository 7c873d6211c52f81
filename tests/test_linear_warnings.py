"""The kernels of the 8-bit-integer products and the gated block read and
write rows of any alignment; the compiler has to know of every such access.
CPU only."""

from __future__ import annotations

import os
import shutil
import subprocess

import pytest

from moe_grouped_gemm_e4m3_amd.build import CSRC, INCLUDE

HIPCC = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"


@pytest.mark.skipif(not os.path.exists(HIPCC), reason="ROCm toolchain not found")
def test_no_access_claims_more_alignment_than_it_has():
    r = subprocess.run([HIPCC, "--offload-arch=gfx950", "-std=c++17", "-fsyntax-only", "-Werror=align-mismatch",
                        "-Werror=division-by-zero", "-I", INCLUDE, "-I", CSRC, os.path.join(CSRC, "linear.hip")],
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-3000:]
